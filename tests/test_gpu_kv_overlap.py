"""Buffers that lie between one another's rows, or on one another as the calls allow it, give what separate ones give."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from tests.test_gpu_kv import DEV, attention_case, ints
from tests.test_gpu_kv_units import FORMS, on_gpu

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


@pytest.mark.parametrize("D,Hq,Hkv,old,new", [f[1:] for f in FORMS], ids=[f[0] for f in FORMS])
def test_attention_in_place(D, Hq, Hkv, old, new):
    """Outputs on the queries, by every kernel, whole and split."""
    q, *cache = on_gpu(attention_case(np.random.default_rng(D), [old, 0, old // 2], [new, new, 1], Hq, Hkv, D, 32))
    lse = torch.empty(q.shape[:2], device=DEV)
    want, wlse = fp8.fp8_kv_attention(q, *cache, lse=lse)
    for _ in range(3):
        x = q.clone()
        got, glse = fp8.fp8_kv_attention(x, *cache, out=x, lse=torch.empty_like(lse))
        assert got is x and torch.equal(x, want) and torch.equal(glse, wlse)


def test_append_of_columns():
    """Keys and values as columns of one buffer, as a fused projection leaves them."""
    x = torch.randn(20, 6, 64, device=DEV).bfloat16()
    a, b = fp8.kv_cache(3, 2, 16, 64, DEV), fp8.kv_cache(3, 2, 16, 64, DEV)
    fp8.fp8_kv_append(x[:, 2:4], x[:, 4:], ints(range(20)), *a)
    fp8.fp8_kv_append(x[:, 2:4].contiguous(), x[:, 4:].contiguous(), ints(range(20)), *b)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    with pytest.raises(fp8.Fp8fgError):
        fp8.fp8_kv_append(x[:, 2:4], x[:, 4:], ints(range(20)), a[0], a[1], a[2], a[1])
