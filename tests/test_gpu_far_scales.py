"""The quantizers at scales so small that FP32 holds few of their bits: RN32(amax / 448) can
then be a third below amax / 448, and the quotients past 448 saturate.  Codes and
scales bit for bit as the oracle's."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import e4m3, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def small_groups(n):
    """n groups of 128 whose maxima lie between 2^-149 and 2^-118, the first ones 448 (k + 0.45) 2^-149."""
    rng = np.random.default_rng(n)
    top = np.concatenate([448.0 * (np.arange(40) + 0.45) * 2.0 ** -149, 2.0 ** rng.uniform(-149, -118, n - 40)])
    x = (top[:, None] * rng.choice([1.0, -1.0, 0.9, -0.5, 0.3, 0.0], (n, 128))).astype(np.float32)
    x[:, 0], x[:, 1] = top, -top
    return x


def same(got, want, what):
    for g, w in zip(got, want):
        g = g.cpu().numpy()
        w = np.asarray(w, g.dtype)
        bad = np.argwhere(g.view(np.uint32) != w.view(np.uint32)) if g.dtype == np.float32 else np.argwhere(g != w)
        assert bad.size == 0, (what, len(bad), bad[:3].tolist(), g[tuple(bad[0])], w[tuple(bad[0])])


def test_activations():
    x = small_groups(1024)
    for K in (128, 64):                                    # whole and partial groups
        v = np.ascontiguousarray(x[:, :K])
        same(fp8.fp8_quant_act_1x128(dev(v)), quant.quant_act_1x128(v), f"rows of {K}")
    wide = np.ascontiguousarray(x.reshape(128, 8 * 128))
    same(fp8.fp8_quant_act_1x128(dev(wide)), quant.quant_act_1x128(wide), "rows of 1024")
    t = np.ascontiguousarray(x.T)
    same(fp8.fp8_quant_act_1x128(dev(t), transpose_out=True), quant.quant_act_1x128_tokenwise(t), "token-wise")


def test_weights():
    x = small_groups(256)
    for blocks in (x[:128], x[128:], np.concatenate([x[:2]] * 64)):
        w = np.tile(blocks, (2, 3)).astype(np.float32)
        w[128:] *= np.float32(0.37)
        for transpose in (False, True):
            same(fp8.fp8_quant_weight_128x128(dev(w), transpose_out=transpose), quant.quant_weight_128x128(w, transpose), f"weight {transpose}")
        same(fp8.fp8_quant_fprop_operands(dev(x), dev(w[:, :128].copy())),
             quant.quant_act_1x128(x) + quant.quant_weight_128x128(w[:, :128].copy()), "both operands")


def test_requantized_activations():
    rng = np.random.default_rng(4)
    q = e4m3.encode(rng.uniform(-448, 448, (128, 128)).astype(np.float32))
    s = (np.arange(128) % 3 * 2.0 ** -149).astype(np.float32)[None]
    same(fp8.fp8_requant_act_tokenwise(dev(q), dev(s)), quant.requant_act_tokenwise(q, s), "requantized")
