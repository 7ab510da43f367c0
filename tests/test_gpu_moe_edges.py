"""The mixture-of-experts operators where FP32's range ends: against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 2.0 ** -24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# logits of the chosen in decreasing order, the largest from -0.5 to -250: the others' own
# scores lie below FP32's normals, below all of FP32, or within it
FADING = [[-79.9, -88.8], [-50.0, -89.0], [-40.0, -88.0, -92.0, -100.0], [-0.5, -1.0, -87.0, -95.0], [-79.0, -79.5, -88.5, -103.0],
          [-86.0, -88.0, -90.0, -92.0], [-120.0, -121.0, -150.0], [-250.0, -250.5, -251.0, -340.0], [3.0, -20.0, -60.0, -80.0]]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("row", FADING, ids=str)
def test_renormalised_sigmoid_weights_keep_their_ratios(row, bf16):
    """Weights and logits' gradients of chosen experts whose scores are far below the largest one's."""
    k = len(row)
    x = np.full((3, 16), -np.inf, np.float32)
    x[:, 2:2 + k] = row
    t = dev(x).to(torch.bfloat16) if bf16 else dev(x)
    vals = t.float().cpu().numpy()
    idx, w = fp8.moe_route(t, k, scale=2.5)
    ridx, rw, _ = moe.route(vals, k, scale=2.5)
    idx, w = idx.cpu().numpy(), w.cpu().numpy()
    assert np.array_equal(idx, ridx)
    # FP32 arguments (x - ms, x) of two exponentials and a few roundings; weights below FP32's normals
    rel = 4 * (moe.exp_error(2 * np.abs(np.array(vals[0, 2:2 + k])).max()) + 32 * EPS)
    assert np.all(np.abs(w - rw) <= rel * np.abs(rw) + 2.0 ** -126), (w[0], rw[0])
    dw = np.zeros((3, k), np.float32)
    dw[0, 0], dw[1, k - 1], dw[2] = 1.0, 1.0, np.linspace(-1, 1, k)
    g = fp8.moe_route_backward(t, dev(idx), dev(dw), scale=2.5).float().cpu().numpy()
    # dx_i = scale p_i (1 - s_i) d_i with d_i a sum over the chosen: each term p_i p_j carries the errors of both weights
    # (the differences keep what 1 / v - s / v^2 would lose in 64 bits where one weight is nearly 1)
    p = rw / 2.5
    ref, size = np.zeros(x.shape), np.zeros(x.shape)
    for r in range(3):
        for i in range(k):
            rest = 1.0 / (1.0 + np.exp(np.float64(vals[r, idx[r, i]])))
            terms = [2.5 * p[r, i] * rest * (float(dw[r, i]) - float(dw[r, j])) * p[r, j] for j in range(k)]
            ref[r, idx[r, i]], size[r, idx[r, i]] = sum(terms), sum(abs(v) for v in terms)
    lim = 2 * rel * size + 2.0 ** -120 + (2.0 ** -8 * np.abs(ref) if bf16 else 0)
    assert np.all(np.abs(g - ref) <= lim), (g, ref)


@pytest.mark.parametrize("T", [5, 5000, 10000])            # both lane counts
def test_choice_among_scores_below_normals(T):
    """Sigmoid logits of -80 to -103 have scores that FP32 still tells apart: the largest are chosen, in order."""
    rng = np.random.default_rng(T)
    E, k = 128, 6
    x = np.full((T, E), -np.inf, np.float32)
    levels = np.arange(-102.0, -79.0, 0.75).astype(np.float32)        # neighbours differ by more than FP32's step at 2^-147
    for t in range(T):
        x[t, rng.permutation(E)[:levels.size]] = levels
    idx, w = fp8.moe_route(dev(x), k)
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), order)
    few = x.copy()
    few[few > -95.0] = -np.inf                                        # scores of 5e-42 and less only
    idx, w = fp8.moe_route(dev(few), k, n_groups=4, topk_groups=2, group_top=1)
    best = few.reshape(T, 4, E // 4).max(axis=2)
    keep = np.argsort(-best, axis=1, kind="stable")[:, :2]
    live = np.zeros((T, 4), bool)
    np.put_along_axis(live, keep, True, axis=1)
    few[~np.repeat(live, E // 4, axis=1)] = -np.inf
    order = np.argsort(-few, axis=1, kind="stable")[:, :k]
    order = np.where(np.isneginf(np.take_along_axis(few, order, axis=1)), -1, order)
    assert np.array_equal(idx.cpu().numpy(), order)


# g, u, dh whose products g u or dh u pass FP32's range while h, dg and du do not, and small rows beside them
HUGE = [(-50.0, 1e38, 1e-3), (-80.0, 3e38, 1e25), (-60.0, -2e38, 1e20), (-30.0, 1e38, 1e8), (5e19, 2e18, 1e-3), (-87.0, 1e38, -1e30)]


@pytest.mark.parametrize("bf16", [False, True])
def test_gate_of_products_past_range(bf16):
    """The gate and its gradients where a product on the way passes FP32's range and the result does not."""
    M, I = 16, 128
    g, u, dh = (np.zeros((M, I), np.float32) for _ in range(3))
    for r, row in enumerate(HUGE):
        g[r], u[r], dh[r] = row
    rng = np.random.default_rng(5)
    g[8:], u[8:], dh[8:] = rng.standard_normal((8, I)), rng.standard_normal((8, I)), rng.standard_normal((8, I))
    x = dev(np.concatenate([g, u], axis=1))
    x = x.to(torch.bfloat16) if bf16 else x
    vals = x.float().cpu().numpy()
    gv, uv = vals[:, :I], vals[:, I:]
    q, s, qc, sc = fp8.fp8_swiglu(x, checkpoint=True)
    h = moe.gate(gv, uv)
    assert np.all(np.abs(h) < 3e38)
    err = moe.exp_error(gv)
    moe.check_quantized(q.cpu().numpy(), s.cpu().numpy(), h, err * np.abs(h), "h")
    t = dev(dh).to(torch.bfloat16) if bf16 else dev(dh)
    dv = t.float().cpu().numpy()
    q, s, qt, st, qh, sh = (v.cpu().numpy() for v in fp8.fp8_swiglu_backward(qc, sc, t))
    v = moe.decode_rows(qc.cpu().numpy(), sc.cpu().numpy())
    (dg, ag), (du, au) = moe.gate_backward(v[:, :I], v[:, I:], dv)
    hb = moe.gate(v[:, :I], v[:, I:])
    err = moe.exp_error(v[:, :I])
    d, a = np.concatenate([dg, du], 1), np.concatenate([ag * err * 2, au * err * 2], 1)
    assert np.all(np.abs(d) < 3e38)
    moe.check_quantized(q, s, d, a, "gradients along the channels")
    moe.check_quantized(qt, st, d.T, a.T, "gradients along the rows")
    moe.check_quantized(qh, sh, hb.T, (err * np.abs(hb)).T, "h along the rows")


def test_dispatch_without_local_experts():
    """A rank that holds no expert: no entry has a row, in whatever memory the outputs come to lie."""
    x = torch.randn(40, 256, device=DEV)
    idx = torch.randint(0, 8, (40, 4), dtype=torch.int32, device=DEV)
    for _ in range(4):
        spoiled = [torch.full(shape, 7, dtype=torch.int32, device=DEV) for shape in ((40, 4), (40, 4), (1,), (1,))]
        torch.cuda.synchronize()
        del spoiled
        q, s, row_of, offsets, counts = fp8.fp8_moe_dispatch_contiguous(x, idx, 0)
        assert q.shape == (0, 256) and s.shape == (2, 0) and counts.shape == (0,)
        assert torch.all(row_of == -1) and offsets.tolist() == [0]
        spoiled = torch.full((40, 4), 7, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        del spoiled
        q, s, masked, mm = fp8.fp8_moe_dispatch_masked(x, idx, 0, 16)
        assert q.shape == (0, 16, 256) and mm.shape == (0,) and torch.all(masked == -1)
        y = torch.full((128, 256), float("nan"), device=DEV)
        assert torch.all(fp8.moe_combine(y, row_of, torch.ones(40, 4, device=DEV)) == 0)


def test_one_expert_from_a_column():
    """One expert's logits, a column whose second stride means nothing: contiguous, strided and transposed."""
    base = torch.randn(1, 40, device=DEV)
    for x in (base.t(), base.t().contiguous(), torch.randn(40, 8, device=DEV)[:, :1]):
        idx, w = fp8.moe_route(x, 1, renormalize=False)
        assert torch.all(idx == 0) and torch.allclose(w, torch.sigmoid(x), rtol=1e-5)
        g = fp8.moe_route_backward(x, idx, torch.ones(40, 1, device=DEV), renormalize=False)
        s = torch.sigmoid(x.double())
        assert torch.allclose(g.double(), s * (1 - s), rtol=1e-5)
    with pytest.raises(ValueError):
        fp8.moe_route(torch.zeros(2, 8, device=DEV).t(), 1)
