"""GPU parity of the mixture-of-experts operators against the CPU oracle.

Choices, rows, codes of exact quantizations and everything else that is a whole
number must be equal; weights, sums and gradients stay within bounds derived
from their FP32 roundings; quantized values that pass through an exponential
within half an E4M3 step of the exact value plus that error."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import gemm, moe, quant
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 2.0 ** -24                 # one FP32 rounding, relative


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def rounded(x, bf16):
    """x as the GPU sees it: (tensor, float32 values)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    t = t.to(torch.bfloat16) if bf16 else t
    return t.to(DEV), t.float().numpy()


def same_bits(a, b):
    return np.array_equal(np.asarray(a, np.float32).view(np.uint32), np.asarray(b, np.float32).view(np.uint32))


def held(err, lim, what):
    bad = np.argwhere(~(np.abs(err) <= lim))
    assert bad.size == 0, f"{what}: {len(bad)} outside, first {bad[:3].tolist()}"


# ---------------------------------------------------------------------------
# routing

ROUTES = [  # T, E, topk, groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (5, 8, 2, 1, 1, 1), (64, 64, 6, 1, 1, 1), (33, 60, 4, 3, 2, 2), (100, 160, 6, 8, 3, 1),
    (130, 256, 8, 8, 4, 2), (7, 37, 16, 1, 1, 1), (3, 16, 16, 4, 4, 2), (21, 512, 10, 1, 1, 1), (9, 1024, 8, 1, 1, 1),
    (17, 1024, 8, 16, 5, 2), (6, 750, 3, 3, 1, 2), (11, 272, 8, 1, 1, 1), (257, 128, 8, 4, 2, 2)]


def route_check(x, vals, bias, topk, ng, tg, top, score, renorm, scale, what):
    idx, w = fp8.moe_route(x, topk, None if bias is None else dev(bias), ng, tg, top, score, renorm, scale)
    ridx, rw, margin = moe.route(vals, topk, bias, ng, tg, top, score, renorm, scale)
    sure = margin > 1e-5
    assert sure.mean() > 0.5, what
    idx, w = host(idx), host(w)
    assert np.array_equal(idx[sure], ridx[sure]), what
    assert np.all((idx >= -1) & (idx < vals.shape[1])), what
    big = np.max(np.where(np.isfinite(vals), np.abs(vals), 0), axis=1, initial=0.0).astype(np.float64)
    # a score: its exponential and division (and the sum); the weight: another division
    lim = 4 * (moe.exp_error(2 * big) + 32 * EPS)[:, None] * np.abs(rw) + 1e-37
    held((w - rw)[sure], lim[sure], what)
    return idx, w


@pytest.mark.parametrize("score", [fp8.SCORE_SOFTMAX, fp8.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,topk,ng,tg,top", ROUTES)
def test_route(T, E, topk, ng, tg, top, score):
    rng = np.random.default_rng(T * 1000 + E)
    for bf16 in (False, True):
        x, vals = rounded(rng.standard_normal((T, E)) * 2, bf16)
        for bias in (None, (rng.standard_normal(E) * 0.1).astype(np.float32)):
            for renorm in (False, True):
                route_check(x, vals, bias, topk, ng, tg, top, score, renorm, 2.5, f"bf16={bf16} bias={bias is not None}")


@pytest.mark.parametrize("score", [fp8.SCORE_SOFTMAX, fp8.SCORE_SIGMOID])
def test_route_masks(score):
    """-inf experts, groups and rows; the type's lowest value is an ordinary logit."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((12, 64)).astype(np.float32)
    x[0] = -np.inf
    x[1, 1:] = -np.inf                                   # one expert left
    x[2, ::2] = -np.inf
    x[3, :48] = -np.inf                                  # one group of four left
    x[4] = np.finfo(np.float32).min                      # all equal: the lowest indices
    x[5, 8:] = np.finfo(np.float32).min
    x[6] = 0.0
    x[7, 16:18] = 3.0
    x[7, 40:48] = 3.0                                    # ties across groups
    for top in (1, 2):
        for renorm in (False, True):
            idx, w = route_check(dev(x), x, None, 8, 4, 2, top, score, renorm, 1.0, f"top={top}")
            assert np.all(idx[0] == -1) and np.all(w[0] == 0)
            assert idx[1].tolist() == [0] + [-1] * 7
            assert idx[4].tolist() == list(range(8)) and idx[6].tolist() == list(range(8))
            assert np.all(np.isfinite(w))
    bias = np.zeros(64, np.float32)
    bias[10] = -np.inf                                   # a bias of -inf leaves an expert out as well
    idx, _ = route_check(dev(x), x, bias, 8, 4, 2, 2, score, True, 1.0, "bias")
    assert not np.any(idx == 10)


def test_route_strides_and_streams():
    rng = np.random.default_rng(9)
    for dtype, pitch in ((torch.float32, 40), (torch.float32, 37), (torch.bfloat16, 64), (torch.bfloat16, 39)):
        full = torch.zeros(50, pitch)
        full[:, :33] = torch.from_numpy(rng.standard_normal((50, 33)).astype(np.float32))
        full = full.to(dtype).to(DEV)
        x = full[:, :33]
        a = fp8.moe_route(x, 4, score=fp8.SCORE_SOFTMAX)
        b = fp8.moe_route(x.contiguous(), 4, score=fp8.SCORE_SOFTMAX)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        dw = torch.randn(50, 4, device=DEV)
        g1 = fp8.moe_route_backward(x, a[0], dw, fp8.SCORE_SOFTMAX, False)
        g2 = fp8.moe_route_backward(x.contiguous(), a[0], dw, fp8.SCORE_SOFTMAX, False)
        assert torch.equal(g1, g2)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c = fp8.moe_route(x, 4, score=fp8.SCORE_SOFTMAX)
        s.synchronize()
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    idx, w = fp8.moe_route(torch.zeros(0, 8, device=DEV), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    with pytest.raises(ValueError):
        fp8.moe_route(torch.zeros(8, 4, device=DEV).t(), 2)
    with pytest.raises(fp8.Fp8fgError):
        fp8.moe_route(torch.zeros(4, 8, device=DEV), 2, n_groups=3)
    with pytest.raises(fp8.Fp8fgError):                    # three groups take the room of four: 4 * 300 > 1024
        fp8.moe_route(torch.zeros(4, 900, device=DEV), 3, n_groups=3, topk_groups=1)


def test_route_weights_of_small_sigmoid_scores():
    """Renormalised sigmoid weights keep their ratios where every chosen score is too small for FP32."""
    x = np.array([[-200.0, -199.0, -np.inf, -200.0], [-85.0, -84.0, -60.0, -np.inf]], np.float32)
    idx, w = fp8.moe_route(dev(x), 2)
    assert host(idx).tolist() == [[0, 1], [2, 1]]          # equal (zero) scores go to the lowest index
    p = np.exp(-1.0)
    assert np.allclose(host(w)[0], [p / (1 + p), 1 / (1 + p)], rtol=1e-5) and np.allclose(host(w)[1], [1, np.exp(-24.0)], rtol=1e-4)
    dw = np.array([[1.0, 0.0], [0.0, 0.0]], np.float32)
    g = host(fp8.moe_route_backward(dev(x), idx, dev(dw)))
    assert np.allclose(g[0], [p / (1 + p) ** 2, -p / (1 + p) ** 2, 0, 0], rtol=1e-5) and np.all(g[1] == 0)


def test_route_softmax_of_small_chosen_scores():
    """Renormalised softmax weights of experts whose scores are too small for FP32."""
    x = np.full((2, 8), -200.0, np.float32)
    x[:, 0] = 0.0                                        # the only large one ...
    bias = np.zeros(8, np.float32)
    bias[0] = -2.0                                       # ... is steered away from
    x[1, 3] = -199.0
    idx, w = fp8.moe_route(dev(x), 2, dev(bias), score=fp8.SCORE_SOFTMAX)
    assert host(idx)[0].tolist() == [1, 2] and host(idx)[1].tolist() == [1, 2]     # scores underflow to equal zeros
    assert np.allclose(host(w)[0], 0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,ng,tg", [(8200, 256, 8, 4), (4100, 128, 4, 2), (8200, 240, 1, 1), (9000, 64, 1, 1)])
def test_route_many_tokens(T, E, ng, tg, dtype):
    """Batches that take other lane counts choose as small batches of the same tokens do."""
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = torch.randn(T, E, generator=g, device=DEV).to(dtype)
    x[T // 2] = -np.inf
    bias = torch.randn(E, generator=g, device=DEV) * 0.05
    for score in (fp8.SCORE_SIGMOID, fp8.SCORE_SOFTMAX):
        idx, w = fp8.moe_route(x, 8, bias, ng, tg, 2, score)
        parts = [fp8.moe_route(x[i:i + 1000], 8, bias, ng, tg, 2, score) for i in range(0, T, 1000)]
        idx2, w2 = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        if score == fp8.SCORE_SIGMOID:
            assert torch.equal(idx, idx2) and torch.equal(w, w2)
        else:                                              # the row's sum is taken in another order
            same = (idx == idx2).all(1)
            assert same.float().mean() > 0.999 and torch.allclose(w[same], w2[same], rtol=1e-5)
        dw = torch.randn(T, 8, generator=g, device=DEV)
        full = fp8.moe_route_backward(x, idx, dw, score)
        part = torch.cat([fp8.moe_route_backward(x[i:i + 1000], idx[i:i + 1000], dw[i:i + 1000], score) for i in range(0, T, 1000)])
        assert torch.equal(full, part)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", [fp8.SCORE_SOFTMAX, fp8.SCORE_SIGMOID])
@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (6, 8, 3), (65, 64, 6), (33, 100, 4), (40, 256, 8), (9, 300, 16), (5, 1024, 8),
                                      (70, 37, 3), (50, 330, 7), (20, 1001, 16)])
def test_route_backward(T, E, topk, score, renorm):
    rng = np.random.default_rng(T + E)
    for bf16 in (False, True):
        x, vals = rounded(rng.standard_normal((T, E)) * 2, bf16)
        if T > 5:
            vals = vals.copy()
            vals[3, ::3] = -np.inf
            vals[4] = -np.inf
            x = dev(vals, x.dtype)
        idx = moe.route(vals, topk, score=score)[0].astype(np.int32)
        dw = rng.standard_normal((T, topk)).astype(np.float32)
        out = host(fp8.moe_route_backward(x, dev(idx), dev(dw), score, renorm, 2.5))
        ref = moe.route_backward(vals, idx, dw, score, renorm, 2.5)
        # each term of the gradient carries the errors of a few exponentials, divisions and a sum over topk
        mag = moe.route_backward(vals, idx, np.abs(dw) * np.sign(1.0), score, False, 2.5)
        s = moe.scores(vals, score)
        total = np.array([max(sum(s[t, e] for e in idx[t] if e >= 0), 1e-300) for t in range(T)])[:, None]
        size = s * 2.5 * (np.abs(dw).sum(axis=1, keepdims=True)) * (2.0 / total if renorm else 2.0)
        lim = np.maximum(np.abs(mag), size) * 8 * (moe.exp_error(16.0) + 64 * EPS) + 1e-37
        if bf16:
            lim = lim + 2.0 ** -8 * np.abs(ref)
        held(out - ref, lim, f"bf16={bf16}")
        if renorm or score == fp8.SCORE_SIGMOID:
            chosen = np.zeros((T, E), bool)
            for t in range(T):
                chosen[t, idx[t][idx[t] >= 0]] = True
            assert np.all(out[~chosen] == 0)
        if renorm and topk == 1:
            assert np.all(out == 0)


# ---------------------------------------------------------------------------
# rows

def entries(rng, T, E, topk, missing=0.1):
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :topk].astype(np.int32)
    idx[rng.random((T, topk)) < missing] = -1
    return idx


DISPATCH = [  # T, H, E, topk, first, G
    (1, 16, 4, 1, 0, 4), (5, 128, 8, 2, 0, 8), (40, 272, 16, 8, 4, 8), (129, 1040, 8, 3, 0, 8), (300, 1024, 256, 8, 0, 256),
    (700, 144, 60, 16, 30, 30), (2500, 128, 8, 2, 0, 8), (3, 7168, 32, 8, 0, 32), (1100, 32, 1, 1, 0, 1),
    (4200, 1024, 32, 8, 0, 32)]     # the last one's rows pass 32 MB: streaming stores


@pytest.mark.parametrize("T,H,E,topk,first,G", DISPATCH)
def test_dispatch_contiguous(T, H, E, topk, first, G):
    rng = np.random.default_rng(T + H)
    idx = entries(rng, T, E, topk)
    row, off, cnt = moe.rows_contiguous(idx, first, G)
    R = fp8.moe_rows_bound(T, topk, G)
    for bf16 in (False, True):
        x, vals = rounded(workloads.activations(rng, T, H, 0.02, 80.0), bf16)
        q0 = torch.full((R, H), 0x55, dtype=torch.uint8, device=DEV)
        s0 = torch.full(((H + 127) // 128, R), 7.0, device=DEV)
        q, s, grow, goff, gcnt = fp8.fp8_moe_dispatch_contiguous(x, dev(idx), G, first, q=q0, s=s0)
        assert np.array_equal(host(grow), row) and np.array_equal(host(goff), off) and np.array_equal(host(gcnt), cnt)
        eq, es = moe.spread(*quant.quant_act_1x128(vals), row, R)
        used = int(off[-1])
        assert np.array_equal(host(q)[:used], eq[:used]) and same_bits(host(s)[:, :used], es[:, :used])
        assert np.all(host(q)[used:] == 0x55) and np.all(host(s)[:, used:] == 7.0)


@pytest.mark.parametrize("T,H,E,topk,first,G", DISPATCH)
def test_dispatch_masked(T, H, E, topk, first, G):
    rng = np.random.default_rng(T + H + 1)
    idx = entries(rng, T, E, topk)
    for M in (4, max(4, T // 2), T):
        row, mm = moe.rows_masked(idx, first, G, M)
        x, vals = rounded(workloads.activations(rng, T, H, 0.02, 80.0), T % 2 == 0)
        q0 = torch.full((G, M, H), 0x55, dtype=torch.uint8, device=DEV)
        s0 = torch.full((G, (H + 127) // 128, M), 7.0, device=DEV)
        q, s, grow, gmm = fp8.fp8_moe_dispatch_masked(x, dev(idx), G, M, first, q=q0, s=s0)
        assert np.array_equal(host(grow), row) and np.array_equal(host(gmm), mm)
        eq, es = moe.spread(*quant.quant_act_1x128(vals), row, G * M)
        eq, es = eq.reshape(G, M, H), es.reshape(-1, G, M).transpose(1, 0, 2)
        q, s = host(q), host(s)
        for g in range(G):
            n = int(mm[g])
            assert np.array_equal(q[g, :n], eq[g, :n]) and same_bits(s[g, :, :n], es[g, :, :n])
            assert np.all(q[g, n:] == 0x55) and np.all(s[g, :, n:] == 7.0)


def test_dispatch_special_entries():
    """Indices far outside, a token twice at one expert, no tokens, no local expert."""
    x = dev(np.arange(64 * 3, dtype=np.float32).reshape(3, 64))
    idx = np.array([[2, 2], [-2 ** 31, 2 ** 31 - 1], [1, 2]], np.int32)
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(x, dev(idx), 2, 1)
    assert host(row).tolist() == [[128, 129], [-1, -1], [0, 130]] and host(cnt).tolist() == [1, 3]
    assert torch.equal(q[128], q[129]) and torch.equal(s[:, 128], s[:, 129])
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(x, dev(idx), 4, 50)
    assert host(off).tolist() == [0] * 5 and host(cnt).tolist() == [0] * 4 and np.all(host(row) == -1)
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(x[:0], dev(idx[:0]), 4)
    assert host(off).tolist() == [0] * 5 and host(cnt).tolist() == [0] * 4 and row.shape == (0, 2)
    q, s, row, mm = fp8.fp8_moe_dispatch_masked(x[:0], dev(idx[:0]), 4, 8)
    assert host(mm).tolist() == [0] * 4
    z = torch.zeros(2, 64, device=DEV)
    z[1, 3] = -0.0
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(z, dev(np.array([[0], [0]], np.int32)), 1)
    assert np.all(host(s)[:, :2] == 0) and host(q)[1, 3] == 0x80 and host(q)[0].max() == 0
    with pytest.raises(fp8.Fp8fgError):
        fp8.fp8_moe_dispatch_contiguous(x, dev(idx), 4, M_total=128)


def test_dispatch_encodes_every_rounding_boundary():
    """Values within two FP32 steps of every boundary between E4M3 codes, at scales from subnormal to near
    overflow, and signed zeros: codes and scales bit for bit."""
    rng = np.random.default_rng(12)
    m = np.concatenate([np.arange(0, 16) / 16 * 2.0 ** -6, *[2.0 ** e * (1 + np.arange(16) / 16) for e in range(-6, 9)]])
    m = m[m < 448]                                         # codes and the midpoints between them
    scales = np.concatenate([2.0 ** rng.uniform(-40, 40, 24), 2.0 ** rng.uniform(-135, -75, 12), 2.0 ** rng.uniform(75, 118, 12), [2.0 ** -149, 1.0]])
    rows = []
    for s in scales.astype(np.float32):
        for shift in range(-2, 3):
            v = (m * np.float64(s)).astype(np.float32)
            v = (v.view(np.int32) + np.int32(shift) * (v > 0).astype(np.int32)).view(np.float32) * rng.choice([-1, 1], m.size).astype(np.float32)
            v = np.concatenate([v, np.zeros(-m.size % 127, np.float32)]).reshape(-1, 127)
            top = np.full((v.shape[0], 1), np.float32(448.0) * s, np.float32)
            rows.append(np.concatenate([top, v], axis=1))
    x = np.concatenate(rows).astype(np.float32)
    x[::7, 5] = -0.0
    x = x[np.all(np.isfinite(x), axis=1)]
    T = x.shape[0]
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(dev(x), dev(np.zeros((T, 1), np.int32)), 1)
    eq, es = quant.quant_act_1x128(x)
    bad = np.argwhere(host(q)[:T] != eq)
    assert bad.size == 0, (len(bad), bad[:3].tolist(), x[tuple(bad[0])], es[0, bad[0][0]])
    assert same_bits(host(s)[:, :T], es)


def test_dispatch_encodes_every_bf16_ratio():
    """BF16 activations: every 8-bit significand against every 8-bit maximum, over E4M3's range and below it."""
    rows = []
    m = np.arange(128, 256, dtype=np.float32)
    for e in range(0, 20):
        v = m * np.float32(2.0 ** -e)
        for part in (v[:64], v[64:]):
            for a in m:
                rows.append(np.concatenate([[a if e else 255.0], part * np.where(np.arange(64) % 2, -1, 1), np.zeros(63)]))
    x = np.array(rows, np.float32) * 2.0 ** -7
    x[5, 70], x[6, 71] = -0.0, np.float32(-2.0 ** -120)
    x[100:200] *= np.float32(2.0 ** -100)                   # scales below 2^-80, and above 2^80
    x[300:400] *= np.float32(2.0 ** 100)
    T = x.shape[0]
    t, vals = rounded(x, True)
    assert np.array_equal(vals, x)
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(t, dev(np.zeros((T, 1), np.int32)), 1)
    eq, es = quant.quant_act_1x128(x)
    assert np.array_equal(host(q)[:T], eq) and same_bits(host(s)[:, :T], es)


def test_dispatch_scales_of_every_kind():
    """Scales RN32(amax / 448) from subnormal maxima to the largest."""
    rng = np.random.default_rng(15)
    bits = np.concatenate([rng.integers(1, 0x7F800000, 20000), rng.integers(1, 0x04000000, 4000), np.arange(1, 2000),
                           0x3F800000 + 1198 * np.arange(7000)]).astype(np.uint32)
    x = np.zeros((bits.size, 16), np.float32)
    x[:, 3] = bits.view(np.float32)
    x[:, 7] = -x[:, 3] * np.float32(0.37)
    T = x.shape[0]
    q, s, row, off, cnt = fp8.fp8_moe_dispatch_contiguous(dev(x), dev(np.zeros((T, 1), np.int32)), 1)
    eq, es = quant.quant_act_1x128(x)
    assert same_bits(host(s)[:, :T], es)
    bad = np.argwhere(host(q)[:T] != eq)
    assert bad.size == 0, (len(bad), bad[:3].tolist(), x[bad[0][0], [3, 7]], host(q)[bad[0][0]], eq[bad[0][0]])


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,topk,R", [(1, 8, 1, 1), (7, 264, 3, 20), (65, 1040, 8, 512), (300, 512, 16, 700), (4, 7168, 8, 40),
                                        (1100, 1032, 8, 500)])     # the last one: four channels per lane for FP32 rows
def test_combine(T, H, topk, R, out):
    rng = np.random.default_rng(T + H)
    row = rng.integers(-1, R, (T, topk)).astype(np.int32)
    row[0] = -1                                            # a token without rows
    if T > 2:
        row[1, 0], row[2, 0] = R + 5, 2 ** 31 - 1          # outside: no row
    w = rng.standard_normal((T, topk)).astype(np.float32)
    for bf16 in (False, True):
        y, vals = rounded(rng.standard_normal((R, H)), bf16)
        for wt in (w, None):
            o = host(fp8.moe_combine(y, dev(row), None if wt is None else dev(wt), out))
            ref, mag = moe.combine(vals, row, wt)
            lim = (topk + 1) * EPS * mag + 1e-40
            if out == torch.bfloat16:
                lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
            held(o - ref, lim, f"bf16={bf16}")
            assert np.all(o[0] == 0)


def test_combine_ignores_rows_without_an_entry():
    """NaN and infinities in padding rows do not reach any token."""
    y = torch.full((128, 64), float("nan"), device=DEV)
    y[3], y[7] = 2.0, float("inf")
    o = host(fp8.moe_combine(y, dev(np.array([[3, -1], [-1, 3]], np.int32)), dev(np.array([[0.5, np.nan], [np.inf, 1.0]], np.float32))))
    assert np.all(o[0] == 1.0) and np.all(o[1] == 2.0)


@pytest.mark.parametrize("T,H,E,topk,first,G", [(1, 16, 4, 1, 0, 4), (40, 272, 16, 8, 4, 8), (129, 1040, 8, 3, 0, 8), (333, 2048, 24, 16, 0, 6),
                                                (5, 7168, 32, 8, 0, 32), (4200, 1024, 32, 8, 0, 32), (4150, 1040, 16, 8, 4, 8),
                                                (260, 1552, 8, 5, 0, 8)])
def test_combine_backward(T, H, E, topk, first, G):
    rng = np.random.default_rng(T * H)
    idx = entries(rng, T, E, topk)
    row, off, cnt = moe.rows_contiguous(idx, first, G)
    R = fp8.moe_rows_bound(T, topk, G)
    w = rng.standard_normal((T, topk)).astype(np.float32)
    w[0, 0] = 0.0
    for db, yb in ((True, True), (False, False), (True, False), (False, True)):
        d, dv = rounded(workloads.activations(rng, T, H, 0.0, 1.0, 1e-3), db)
        y, yv = rounded(rng.standard_normal((R, H)), yb)
        q0 = torch.full((R, H), 0x55, dtype=torch.uint8, device=DEV)
        s0 = torch.full(((H + 127) // 128, R), 7.0, device=DEV)
        args = (d, y, dev(row.astype(np.int32)), dev(w), dev(off.astype(np.int32)), dev(cnt.astype(np.int32)))
        q, s, dw = fp8.fp8_moe_combine_backward(*args, q=q0, s=s0)
        eq, es = moe.spread(*quant.quant_act_1x128(dv), row, R, w)
        used = int(off[-1])
        assert np.array_equal(host(q)[:used], eq[:used]) and same_bits(host(s)[:, :used], es[:, :used])
        assert np.all(host(q)[used:] == 0x55) and np.all(host(s)[:, used:] == 7.0)
        ref, mag = moe.combine_dw(dv, yv, row)
        held(host(dw) - ref, H * EPS * mag, "dw")
        dw2 = fp8.fp8_moe_combine_backward(*args)[2]
        assert torch.equal(dw, dw2)                        # the same bits every time


# ---------------------------------------------------------------------------
# the gate

def gate_error(g, u):
    """h's relative error, and a sigmoid below FP32's normal range that may flush to zero."""
    return moe.exp_error(g) * np.abs(moe.gate(g, u)) + 2.0 ** -126 * np.abs(g.astype(np.float64) * u)


@pytest.mark.parametrize("M,I", [(1, 128), (31, 128), (33, 256), (300, 384), (129, 2048)])
@pytest.mark.parametrize("bf16", [False, True])
def test_swiglu(M, I, bf16):
    rng = np.random.default_rng(M + I)
    x = workloads.activations(rng, M, 2 * I, 0.01, 30.0, 2.0)
    x[0, :I] = -90.0                                       # sigmoid near and past underflow
    if M > 1:
        x[1, :I] = 90.0
        x[M - 1] = 0.0
    gu, vals = rounded(x, bf16)
    g, u = vals[:, :I], vals[:, I:]
    h = moe.gate(g, u)
    for used in (None, M, M // 2, 0):
        rows = None if used is None else torch.tensor([used], dtype=torch.int32, device=DEV)
        n = M if used is None else used
        bufs = [torch.full(s, v, dtype=t, device=DEV) for s, v, t in (((M, I), 0x55, torch.uint8), ((I // 128, M), 7.0, torch.float32),
                                                                      ((M, 2 * I), 0x55, torch.uint8), ((2 * I // 128, M), 7.0, torch.float32))]
        q, s, qc, sc = fp8.fp8_swiglu(gu, rows, True, *bufs)
        q2, s2 = fp8.fp8_swiglu(gu, rows, q=bufs[0].clone(), s=bufs[1].clone())
        assert torch.equal(q, q2) and torch.equal(s, s2)
        q, s, qc, sc = host(q), host(s), host(qc), host(sc)
        moe.check_quantized(q[:n], s[:, :n], h[:n], gate_error(g[:n], u[:n]), "h")
        eq, es = quant.quant_act_1x128(vals)
        assert np.array_equal(qc[:n], eq[:n]) and same_bits(sc[:, :n], es[:, :n])
        assert np.all(q[n:] == 0x55) and np.all(qc[n:] == 0x55) and np.all(s[:, n:] == 7.0) and np.all(sc[:, n:] == 7.0)


def test_swiglu_masked():
    rng = np.random.default_rng(2)
    G, M, I = 5, 70, 256
    mm = np.array([0, 70, 1, 33, 64], np.int32)
    gu, vals = rounded(rng.standard_normal((G, M, 2 * I)) * 2, True)
    gu[0] = float("nan")                                   # rows that are not read
    q0 = torch.full((G, M, I), 0x55, dtype=torch.uint8, device=DEV)
    s0 = torch.full((G, I // 128, M), 7.0, device=DEV)
    q, s = fp8.fp8_swiglu(gu, dev(mm), q=q0, s=s0)
    for g in range(G):
        n = mm[g]
        a, b = fp8.fp8_swiglu(gu[g].contiguous())
        assert torch.equal(q[g, :n], a[:n]) and torch.equal(s[g, :, :n], b[:, :n])
        assert torch.all(q[g, n:] == 0x55) and torch.all(s[g, :, n:] == 7.0)
    v = vals[1]
    moe.check_quantized(host(q[1]), host(s[1]), moe.gate(v[:, :I], v[:, I:]),
                        gate_error(v[:, :I], v[:, I:]), "masked")


@pytest.mark.parametrize("M,I", [(16, 128), (128, 128), (144, 256), (400, 384), (128, 2048)])
@pytest.mark.parametrize("bf16", [False, True])
def test_swiglu_backward(M, I, bf16):
    rng = np.random.default_rng(M * I)
    x = workloads.activations(rng, M, 2 * I, 0.01, 20.0, 2.0)
    x[2, :] = 0.0
    qc, sc = quant.quant_act_1x128(x)
    dh, dv = rounded(workloads.activations(rng, M, I, 0.0, 1.0, 1e-3), bf16)
    v = moe.decode_rows(qc, sc)
    g, u = v[:, :I], v[:, I:]
    nb = I // 128
    for used in (None, M, max(M - 5, 1), M // 2):
        n = M if used is None else used
        rows = None if used is None else torch.tensor([n], dtype=torch.int32, device=DEV)
        shapes = ((M, 2 * I), (2 * nb, M), (2 * I, M), (-(-M // 128), 2 * I), (I, M), (-(-M // 128), I))
        bufs = [torch.full(s, 7.0 if k % 2 else 0x55, dtype=torch.float32 if k % 2 else torch.uint8, device=DEV)
                for k, s in enumerate(shapes)]
        q, s, qt, st, qh, sh = (host(t) for t in fp8.fp8_swiglu_backward(dev(qc), dev(sc), dh, rows, out=bufs))
        live = (np.arange(M) < n)[:, None]
        (dg, ag), (du, au) = moe.gate_backward(g, u, np.where(live, dv, 0.0))
        h = np.where(live, moe.gate(g, u), 0.0)
        err = moe.exp_error(g)
        d, a = np.concatenate([dg, du], 1), np.concatenate([ag * err * 2, au * err * 2], 1)
        a = a + 2.0 ** -126 * np.tile(np.abs(dv) * (1 + np.abs(g)) * (1 + np.abs(u)), 2)
        moe.check_quantized(q[:n], s[:, :n], d[:n], a[:n], "rows")
        assert np.all(q[n:] == 0x55) and np.all(s[:, n:] == 7.0)
        done = min(M, -(-n // 128) * 128)                  # whole 128-row groups
        moe.check_quantized(qt[:, :done], st[: -(-n // 128)], d.T[:, :done], a.T[:, :done], "columns")
        moe.check_quantized(qh[:, :done], sh[: -(-n // 128)], h.T[:, :done], gate_error(g, u).T[:, :done], "h")
        assert np.all(qt[:, done:] == 0x55) and np.all(qh[:, done:] == 0x55)
        assert np.all(st[-(-n // 128):] == 7.0) and np.all(sh[-(-n // 128):] == 7.0)


@pytest.mark.parametrize("bf16", [False, True])
def test_gate_large(bf16):
    """Outputs past 32 MB (streaming stores): the bits of small calls on the same rows."""
    M, I = 6144, 2048
    g = torch.Generator(device=DEV).manual_seed(3)
    dtype = torch.bfloat16 if bf16 else torch.float32
    gu = (torch.randn(M, 2 * I, generator=g, device=DEV) * 2).to(dtype)
    dh = torch.randn(M, I, generator=g, device=DEV).to(dtype)
    q, s, qc, sc = fp8.fp8_swiglu(gu, checkpoint=True)
    big = fp8.fp8_swiglu_backward(qc, sc, dh)
    for lo in (0, 2048, M - 256):
        k = slice(lo, lo + 256)
        a = fp8.fp8_swiglu(gu[k].contiguous(), checkpoint=True)
        for t, u in zip((q[k], s[:, k], qc[k], sc[:, k]), a):
            assert torch.equal(t, u)
        b = fp8.fp8_swiglu_backward(qc[k].contiguous(), sc[:, k].contiguous(), dh[k].contiguous())
        kb = slice(lo // 128, lo // 128 + 2)
        for t, u in zip((big[0][k], big[1][:, k], big[2][:, k], big[3][kb], big[4][:, k], big[5][kb]), b):
            assert torch.equal(t, u)


# ---------------------------------------------------------------------------
# the experts' weight gradients

def operand(rng, n, R, sigma):
    return quant.quant_act_1x128(workloads.activations(rng, n, R, 0.01, 40.0, sigma))


@pytest.mark.parametrize("M,N", [(256, 256), (300, 512), (16, 256), (1, 256), (144, 208), (128, 384), (272, 16)])
def test_wgrad(M, N):
    rng = np.random.default_rng(M + N)
    off = np.array([0, 128, 128, 512, 640], np.int32)      # the second expert has no rows
    R = 896                                                # the last 256 belong to nobody
    qa, sa = operand(rng, M, R, 1e-3)
    qb, sb = operand(rng, N, R, 1.0)
    qa[:, 640:], qb[:, 640:] = 0x7F, 0x7F                  # NaN codes: never read into a result
    sa[640 // 128:], sb[640 // 128:] = np.nan, np.nan
    sa[0, M // 2] = 0.0                                    # a zero group over nonzero codes
    a, b = (dev(qa), dev(sa)), (dev(qb), dev(sb))
    out = torch.full((4, M, N), float("nan"), device=DEV)
    c = fp8.fp8_grouped_gemm_wgrad(*a, *b, dev(off), out=out)
    c = host(c)
    start = rng.standard_normal((4, M, N)).astype(np.float32)
    more = host(fp8.fp8_grouped_gemm_wgrad(*a, *b, dev(off), out=dev(start), accumulate=True))
    for g in range(4):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            assert np.all(c[g] == 0) and np.array_equal(more[g], start[g])
            continue
        ref, mag = gemm.gemm_blockscaled_ref(qa[:, lo:hi], sa[lo // 128:hi // 128], qb[:, lo:hi], sb[lo // 128:hi // 128], "1x128")
        held(c[g] - ref, gemm.U * mag, f"expert {g}")
        held(more[g] - (ref + start[g]), gemm.U * mag + 2 * EPS * (np.abs(ref) + np.abs(start[g])), f"expert {g} accumulated")


def check_experts(c, qa, sa, qb, sb, off, rng, start=None):
    """Every expert's result on some of its rows, whole where it has no rows."""
    M = qa.shape[0]
    for g in range(len(off) - 1):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            assert np.all(c[g] == (0 if start is None else start[g]))
            continue
        rows = np.unique(np.concatenate([np.arange(min(M, 3)), rng.integers(0, M, 24), np.arange(max(M - 3, 0), M)]))
        ref, mag = gemm.gemm_blockscaled_ref(qa[:, lo:hi], sa[lo // 128:hi // 128], qb[:, lo:hi], sb[lo // 128:hi // 128], "1x128", rows=rows)
        lim = gemm.U * mag
        if start is not None:
            ref = ref + start[g][rows]
            lim = lim + 4 * EPS * (np.abs(ref) + np.abs(start[g][rows]))
        held(c[g][rows] - ref, lim, f"expert {g}")


@pytest.mark.parametrize("M,N", [(1000, 1024), (1024, 1024), (1024, 1040)])
def test_wgrad_large_tiles(M, N):
    """Over 256 tiles of 256 x 256: one expert longer than an accumulator takes, several short ones, some empty."""
    rng = np.random.default_rng(M + N)
    blocks = np.array([1, 0, 2, 70, 1, 3, 0, 1, 2, 1, 1, 4, 1, 0, 1, 2, 1, 1, 64, 1])
    off = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32) * 128
    R = int(off[-1]) + 256
    qa, sa = operand(rng, M, R, 1e-3)
    qb, sb = operand(rng, N, R, 1.0)
    qa[:, off[-1]:], qb[:, off[-1]:] = 0x7F, 0x7F
    args = (dev(qa), dev(sa), dev(qb), dev(sb), dev(off))
    G = len(blocks)
    c = fp8.fp8_grouped_gemm_wgrad(*args, out=torch.full((G, M, N), float("nan"), device=DEV))
    check_experts(host(c), qa, sa, qb, sb, off, rng)
    start = rng.standard_normal((G, M, N)).astype(np.float32)
    more = fp8.fp8_grouped_gemm_wgrad(*args, out=dev(start), accumulate=True)
    check_experts(host(more), qa, sa, qb, sb, off, rng, start)
    if N % 256 == 0:                                       # the dense call's bits, up to 64 K-blocks
        for g in (2, 11, 18):
            k, kb = slice(off[g], off[g + 1]), slice(off[g] // 128, off[g + 1] // 128)
            d = fp8.fp8_gemm_blockscaled(dev(qa[:, k]), dev(sa[kb]), dev(qb[:, k]), dev(sb[kb]), fp8.BSCALE_1x128, torch.float32)
            assert torch.equal(c[g], d)


def test_wgrad_many_experts_large_tiles():
    """Over 64 experts and over 256 tiles: the natural order of the experts."""
    rng = np.random.default_rng(16)
    G, M, N = 80, 512, 512
    blocks = rng.integers(0, 3, G)
    off = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32) * 128
    qa, sa = operand(rng, M, int(off[-1]), 1e-3)
    qb, sb = operand(rng, N, int(off[-1]), 1.0)
    c = host(fp8.fp8_grouped_gemm_wgrad(dev(qa), dev(sa), dev(qb), dev(sb), dev(off)))
    check_experts(c, qa, sa, qb, sb, off, rng)


@pytest.mark.parametrize("N", [256, 128])
def test_wgrad_long_contraction(N):
    """More rows than one accumulator takes (64 K-blocks): several pieces, also when accumulating."""
    rng = np.random.default_rng(N)
    M, R = 40, 128 * 140
    off = np.array([0, 128 * 64, 128 * 64 + 128, R], np.int32)
    qa, sa = operand(rng, M, R, 1e-3)
    qb, sb = operand(rng, N, R, 1.0)
    start = rng.standard_normal((3, M, N)).astype(np.float32)
    args = (dev(qa), dev(sa), dev(qb), dev(sb), dev(off))
    c = host(fp8.fp8_grouped_gemm_wgrad(*args))
    more = host(fp8.fp8_grouped_gemm_wgrad(*args, out=dev(start), accumulate=True))
    for g in range(3):
        lo, hi = off[g], off[g + 1]
        ref, mag = gemm.gemm_blockscaled_ref(qa[:, lo:hi], sa[lo // 128:hi // 128], qb[:, lo:hi], sb[lo // 128:hi // 128], "1x128")
        held(c[g] - ref, gemm.U * mag, f"expert {g}")
        held(more[g] - (ref + start[g]), gemm.U * mag + 4 * EPS * (np.abs(ref) + np.abs(start[g])), f"expert {g} accumulated")


def test_wgrad_many_experts_and_offsets_out_of_range():
    """Over 64 experts (the natural order); offsets past the end are clamped, unaligned ones rounded down."""
    rng = np.random.default_rng(6)
    G, M, N = 70, 32, 256
    R = 128 * G
    off = (128 * np.arange(G + 1)).astype(np.int32)
    qa, sa = operand(rng, M, R, 1e-3)
    qb, sb = operand(rng, N, R, 1.0)
    args = (dev(qa), dev(sa), dev(qb), dev(sb))
    c = host(fp8.fp8_grouped_gemm_wgrad(*args, dev(off)))
    for g in (0, 33, 69):
        k = slice(128 * g, 128 * g + 128)
        ref, mag = gemm.gemm_blockscaled_ref(qa[:, k], sa[g:g + 1], qb[:, k], sb[g:g + 1], "1x128")
        held(c[g] - ref, gemm.U * mag, f"expert {g}")
    odd = np.array([-5, 130, 100000, 7], np.int32)         # clamped to [0, 128), [128, R), nothing
    c = host(fp8.fp8_grouped_gemm_wgrad(*args, dev(odd)))
    for g, (lo, hi) in enumerate(((0, 128), (128, R))):
        ref, mag = gemm.gemm_blockscaled_ref(qa[:, lo:hi], sa[lo // 128:hi // 128], qb[:, lo:hi], sb[lo // 128:hi // 128], "1x128")
        held(c[g] - ref, gemm.U * mag, f"expert {g}")
    assert np.all(c[2] == 0)


# ---------------------------------------------------------------------------
# capture

def test_decode_path_in_a_graph():
    """Route, dispatch, gate and combine captured once and replayed with new inputs, eager work in between."""
    T, E, H, I, M = 24, 16, 256, 128, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.randn(T, E, generator=g, device=DEV)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    gu = torch.randn(E, M, 2 * I, generator=g, device=DEV).bfloat16()

    def step():
        idx, w = fp8.moe_route(logits, 4, score=fp8.SCORE_SOFTMAX, n_groups=4, topk_groups=2)
        q, s, row, mm = fp8.fp8_moe_dispatch_masked(x, idx, E, M)
        h, hs = fp8.fp8_swiglu(gu, mm)
        return idx, w, row, mm, fp8.moe_combine(gu, row, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        logits.copy_(torch.randn(T, E, generator=g, device=DEV))
        gu.copy_(torch.randn(E, M, 2 * I, generator=g, device=DEV))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b), k
