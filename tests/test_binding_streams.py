"""The stream that the binding passes on is the current one of the tensor's device."""
import pytest
import torch

import fp8_fine_grained_amd as fp8


class OnDevice:
    device = "cuda:3"

    def get_device(self):
        return 3


def test_without_torchs_private_entry(monkeypatch):
    """The public call serves where torch lacks the handle's own entry."""
    class Stream:
        cuda_stream = 77

    seen = []
    monkeypatch.setattr(fp8, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: seen.append(device) or Stream())
    assert fp8._stream(OnDevice()) == 77 and seen == ["cuda:3"]


def test_through_the_entry(monkeypatch):
    monkeypatch.setattr(fp8, "_raw_stream", lambda index: 100 + index)
    assert fp8._stream(OnDevice()) == 103


@pytest.mark.gpu
def test_handles_agree(monkeypatch):
    x = torch.zeros(4, 128, device="cuda")
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            fast = fp8._stream(x)
            with monkeypatch.context() as m:
                m.setattr(fp8, "_raw_stream", None)
                assert fp8._stream(x) == fast == stream.cuda_stream
