"""Weight gradients on every tile that their sizes choose, against the 64-bit oracle and the dense call."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import gemm, quant
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def operand(rng, n, R, sigma):
    return quant.quant_act_1x128(workloads.activations(rng, n, R, 0.01, 40.0, sigma))


def held(c, qa, sa, qb, sb, lo, hi, rows, what, start=None):
    """|c - c*| <= 2^-14 S on some rows (plus the additions to what was there, one per 64 K-blocks)."""
    ref, mag = gemm.gemm_blockscaled_ref(qa[:, lo:hi], sa[lo // 128:hi // 128], qb[:, lo:hi], sb[lo // 128:hi // 128], "1x128", rows=rows)
    lim = gemm.U * mag
    if start is not None:
        ref = ref + start[rows]
        lim = lim + ((hi - lo) // 8192 + 2) * 2.0 ** -24 * (mag + np.abs(start[rows]))
    bad = np.argwhere(~(np.abs(c[rows] - ref) <= lim))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist())


@pytest.mark.parametrize("G,M,N", [(1, 2048, 4096), (2, 2048, 4096), (1, 1999, 7168)])
def test_one_expert_filling_half_the_chip_runs_the_dense_calls_tiles(G, M, N):
    """128 and more 256 x 256 tiles to an expert: the bits of the dense Wgrad call, which runs those tiles."""
    rng = np.random.default_rng(G + N)
    off = np.array([0, 384, 640], np.int32)[:G + 1]
    R = int(off[-1])
    qa, sa = operand(rng, M, R, 1e-3)
    qb, sb = operand(rng, N, R, 1.0)
    c = fp8.fp8_grouped_gemm_wgrad(dev(qa), dev(sa), dev(qb), dev(sb), dev(off))
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        k, kb = slice(lo, hi), slice(lo // 128, hi // 128)
        d = fp8.fp8_gemm_blockscaled(dev(qa[:, k]), dev(sa[kb]), dev(qb[:, k]), dev(sb[kb]), fp8.BSCALE_1x128, torch.float32)
        assert torch.equal(c[g], d), g
        held(c[g].cpu().numpy(), qa, sa, qb, sb, lo, hi, np.array([0, 700, M - 1]), f"expert {g}")
