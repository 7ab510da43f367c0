"""Writes into pages whose scale so far is any FP32 number, as a cache that other code began may have it."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import e4m3, kv
from tests.test_gpu_kv import dev, host, ints, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("was", [0.3, 0.7071, 3.14159e-3, 1.9999999, 2.0 ** -130, 1.1 * 2.0 ** -127, 1.5 * 2.0 ** -126, 1.7 * 2.0 ** 120, 1.3 * 2.0 ** 127])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_under_any_scale(was, bf16):
    """Single tokens, short and long runs; values below, about and above the scale's."""
    rng = np.random.default_rng(7)
    was = float(np.float32(was))
    slots = [5] + [64 + 3 + i for i in range(9)] + [128 + 1 + i for i in range(40)] + [196] + [260 + i for i in range(60)]
    for grow in (1.0, 30 * was, 100 * was, 1e-3 * was, 0.0):
        if 0.0 < grow < 1e36:
            run_append(rng, len(slots), slots, 2, 128, 64, 6, bf16, grow, was)
    run_append(rng, len(slots), slots, 2, 128, 64, 6, bf16, 0.0, was)


def test_append_at_the_middles_between_codes():
    """Quotients next to the middle of two codes, where a product with the rounded inverse takes the wrong one."""
    rng = np.random.default_rng(8)
    c = e4m3.decode(np.arange(0, 0x7E, dtype=np.uint8)).astype(np.float64)
    for _ in range(20):
        s = np.float32(rng.uniform(0.5, 1.0))
        mid = ((c[:-1] + c[1:]) / 2 * float(s)).astype(np.float32)
        x = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), mid])[:384].reshape(3, 1, 128)
        x = np.minimum(x, np.float32(223.0))                  # the scale stays: 448 / 2 < 224
        kc, vc, sc = np.zeros((1, 1, 16, 128), np.uint8), np.zeros((1, 1, 128, 16), np.uint8), np.full((1, 1), s, np.float32)
        t, gpu = dev(x), [dev(kc), dev(sc), dev(vc), dev(sc)]
        fp8.fp8_kv_append(t, t, ints([4, 5, 6]), *gpu)
        want, ws = kv.append(x, [4, 5, 6], kc, sc, 16)
        assert np.array_equal(host(gpu[1]), ws) and np.array_equal(host(gpu[3]), ws) and ws[0, 0] == s
        assert np.array_equal(host(gpu[0]), want) and np.array_equal(host(gpu[2]), want.transpose(0, 1, 3, 2))
        for i in range(3):                                     # one token at a time
            fp8.fp8_kv_append(t[i:i + 1], t[i:i + 1], ints([8 + i]), *gpu)
        assert np.array_equal(host(gpu[0])[0, 0, 8:11], want[0, 0, 4:7]) and torch.equal(gpu[2][..., 8:11], gpu[2][..., 4:7])
