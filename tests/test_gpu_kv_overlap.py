"""Buffers that lie between one another's rows, or on one another as the calls allow it, give what separate ones give."""
import pytest
import torch

import fp8_fine_grained_amd as fp8
from tests.test_gpu_kv import DEV, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 33])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_between_rows(T, dtype):
    """Inputs and outputs as columns of one buffer; queries in place and keys elsewhere in it; keys in place."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, 14, 64, generator=g, device=DEV).to(dtype)
    pos, (freqs, _) = ints(range(5, 5 + T)), fp8.rope_frequencies(64, device=DEV)
    q, k = fp8.rope(x[:, :4].contiguous(), x[:, 4:6].contiguous(), pos, freqs)
    y = x.clone()
    fp8.rope(y[:, :4], y[:, 4:6], pos, freqs, q_out=y[:, 6:10], k_out=y[:, 11:13])
    assert torch.equal(y, torch.cat([x[:, :6], q, x[:, 10:11], k, x[:, 13:]], 1))
    y = x.clone()
    fp8.rope(y[:, :4], y[:, 4:6], pos, freqs, q_out=y[:, :4], k_out=y[:, 8:10])
    assert torch.equal(y, torch.cat([q, x[:, 4:8], k, x[:, 10:]], 1))
    y = x.clone()
    out, _ = fp8.rope(y[:, :4], y[:, 4:6], pos, freqs, k_out=y[:, 4:6])
    assert torch.equal(out, q) and torch.equal(y, torch.cat([x[:, :4], k, x[:, 6:]], 1))
    with pytest.raises(fp8.Fp8fgError):
        fp8.rope(y[:, :4], y[:, 4:6], pos, freqs, q_out=y[:, 1:5])
