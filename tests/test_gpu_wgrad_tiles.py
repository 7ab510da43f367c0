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


def codes(rng, n, R):
    """Random codes (no NaN) and scales over 2^16, one group in fifty with scale 0."""
    q = rng.integers(0, 0x7F, (n, R), dtype=np.uint8) | rng.choice(np.array([0, 0x80], np.uint8), (n, R))
    s = np.exp2(rng.uniform(-16, 0, (R // 128, n))).astype(np.float32)
    s[rng.random(s.shape) < 0.02] = 0.0
    return q, s


def test_wide_tiles_in_many_pieces():
    """More than 256 wide tiles; experts of 63 to 193 K-blocks, one to four pieces of 64, and scales of 0 at their edges."""
    rng = np.random.default_rng(21)
    blocks = np.array([128, 0, 129, 1, 140, 64, 2, 193, 63, 65] + [1, 0] * 17)
    off = (np.concatenate([[0], np.cumsum(blocks)]) * 128).astype(np.int32)
    G, M, N, R = len(blocks), 500, 768, int(off[-1]) + 128
    (qa, sa), (qb, sb) = codes(rng, M, R), codes(rng, N, R)
    for g in (0, 2, 4, 7):                                 # groups of 0 at the ends of pieces
        first = off[g] // 128
        sa[[first, first + 63, first + 64, first + 127], 3] = 0.0
        sb[[first + 63, first + 64], 5] = 0.0
    qa[:, off[-1]:], qb[:, off[-1]:] = 0x7F, 0x7F
    args = tuple(map(dev, (qa, sa, qb, sb, off)))
    c = fp8.fp8_grouped_gemm_wgrad(*args, out=torch.full((G, M, N), float("nan"), device=DEV))
    assert torch.equal(c, fp8.fp8_grouped_gemm_wgrad(*args))
    start = torch.randn(G, M, N, device=DEV)
    more = fp8.fp8_grouped_gemm_wgrad(*args, out=start.clone(), accumulate=True)
    rows = np.array([0, 3, 255, 256, 499])
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            assert torch.all(c[g] == 0) and torch.equal(more[g], start[g])
            continue
        held(c[g].cpu().numpy(), qa, sa, qb, sb, lo, hi, rows, f"expert {g}")
        held(more[g].cpu().numpy(), qa, sa, qb, sb, lo, hi, rows, f"expert {g} accumulated", start[g].cpu().numpy())
