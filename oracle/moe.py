"""The mixture-of-experts operators, from their definitions (test infrastructure only).

Plain loops over tokens and entries, in float64 except where the method fixes
a float32 step; quantized rows come in from ``oracle.quant``.  The choice of experts, the rows of the two grouped layouts,
the weighted sum of the rows, the gate and every gradient are written out from
their formulas; nothing here is shared with the HIP library.
"""

import numpy as np

from . import e4m3

SOFTMAX, SIGMOID = 0, 1


def scores(x, score):
    """Scores of float rows x [T][E] in float64; a row of -inf has softmax scores 0."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        m = np.max(x, axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isinf(m), 0.0, m))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total > 0, total, 1.0)


def route(x, topk, bias=None, n_groups=1, topk_groups=1, group_top=1, score=SIGMOID, renormalize=True, scale=1.0):
    """(idx [T][topk], w float64 [T][topk], margin [T]): margin is the smallest
    relative distance between two scores that the choice compares, over the ties
    of equal scores (which go to the lowest index whatever the rounding)."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    s = scores(x, score)
    c = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
    c = np.where(np.isneginf(x), -np.inf, c)
    per = E // n_groups
    idx = np.full((T, topk), -1, dtype=np.int64)
    w = np.zeros((T, topk))
    margin = np.full(T, np.inf)

    def closest(order, value, take):
        best = np.inf
        for a, b in zip(order[:take], order[1:take + 1]):
            if value[a] != value[b]:
                best = min(best, (value[a] - value[b]) / max(abs(value[a]), abs(value[b])))
        return best

    for t in range(T):
        groups = list(range(n_groups))
        if topk_groups < n_groups:
            gs = {}
            for g in groups:
                live = sorted((v for v in c[t, g * per:(g + 1) * per] if v > -np.inf), reverse=True)
                if live:
                    gs[g] = sum(live[:group_top])
            order = sorted(gs, key=lambda g: (-gs[g], g))
            margin[t] = min(margin[t], closest(order, gs, topk_groups))
            groups = order[:topk_groups]
        pool = [e for g in groups for e in range(g * per, (g + 1) * per) if c[t, e] > -np.inf]
        pool.sort(key=lambda e: (-c[t, e], e))
        margin[t] = min(margin[t], closest(pool, c[t], topk))
        chosen = pool[:topk]
        idx[t, :len(chosen)] = chosen
        if not chosen:
            continue
        v = s[t, chosen]
        if renormalize:                          # through logarithms: scores may be too small to represent
            log = x[t, chosen] - (np.logaddexp(0.0, x[t, chosen]) if score == SIGMOID else 0.0)
            v = np.exp(log - np.max(log))
            v = v / v.sum()
        w[t, :len(chosen)] = scale * v
    return idx, w, margin


def route_backward(x, idx, dw, score=SIGMOID, renormalize=True, scale=1.0):
    """dL/dx float64 [T][E] for the fixed choice idx, by the chain rule through s."""
    s = scores(x, score)
    T, E = s.shape
    dx = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        ds = np.zeros(E)
        total = sum(s[t, idx[t, j]] for j in slots)
        for j in slots:
            if renormalize:
                if total == 0:
                    continue
                # w_j = scale s_j / total
                ds[idx[t, j]] += scale * dw[t, j] / total
                for i in slots:
                    ds[idx[t, i]] -= scale * dw[t, j] * s[t, idx[t, j]] / total ** 2
            else:
                ds[idx[t, j]] += scale * dw[t, j]
        if score == SIGMOID:
            dx[t] = ds * s[t] * (1.0 - s[t])
        else:
            dx[t] = s[t] * (ds - np.dot(ds, s[t]))
    return dx


def rows_contiguous(idx, first, G):
    """(row_of, offsets, counts): entries in order, each expert's rows padded to 128."""
    flat = np.asarray(idx).reshape(-1)
    counts = np.array([int(np.sum(flat == first + g)) for g in range(G)], dtype=np.int64)
    offsets = np.concatenate([[0], np.cumsum(-(-counts // 128) * 128)]).astype(np.int64)
    row, seen = np.full(flat.size, -1, dtype=np.int64), [0] * G
    for i, e in enumerate(flat):
        g = int(e) - first
        if 0 <= g < G:
            row[i] = offsets[g] + seen[g]
            seen[g] += 1
    return row.reshape(np.shape(idx)), offsets, counts


def rows_masked(idx, first, G, m_max):
    """(row_of, masked_m) of the masked layout; entries past m_max have no row."""
    flat = np.asarray(idx).reshape(-1)
    row, seen = np.full(flat.size, -1, dtype=np.int64), [0] * G
    for i, e in enumerate(flat):
        g = int(e) - first
        if 0 <= g < G:
            if seen[g] < m_max:
                row[i] = g * m_max + seen[g]
            seen[g] += 1
    return row.reshape(np.shape(idx)), np.minimum(seen, m_max).astype(np.int64)


def spread(q, s, row_of, R, w=None):
    """Token codes q [T][H] and scales s [H/128][T] in their rows ([R][H], [H/128][R]),
    zero elsewhere; with w the scales times |w| (one float32 product) and the
    codes' signs times w's."""
    qo = np.zeros((R, q.shape[1]), np.uint8)
    so = np.zeros((s.shape[0], R), np.float32)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            r = row_of[t, j]
            if r < 0:
                continue
            qo[r] = q[t]
            so[:, r] = s[:, t]
            if w is not None:
                so[:, r] = s[:, t] * np.float32(abs(w[t, j]))
                if w[t, j] < 0:
                    qo[r] = q[t] ^ 0x80
    return qo, so


def combine(y, row_of, w=None):
    """(sum_j w_tj y[row_tj], sum_j |w_tj y[row_tj]|) in float64."""
    y = np.asarray(y, dtype=np.float64)
    T, k = row_of.shape
    out, mag = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= row_of[t, j] < y.shape[0]:
                v = (1.0 if w is None else float(w[t, j])) * y[row_of[t, j]]
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def combine_dw(dout, y, row_of):
    """(<dout_t, y[row_tj]>, the same of magnitudes), 0 without a row."""
    dout, y = np.asarray(dout, dtype=np.float64), np.asarray(y, dtype=np.float64)
    dw, mag = np.zeros(row_of.shape), np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            if 0 <= row_of[t, j] < y.shape[0]:
                p = dout[t] * y[row_of[t, j]]
                dw[t, j], mag[t, j] = p.sum(), np.abs(p).sum()
    return dw, mag


def gate(g, u):
    """h = g sigmoid(g) u in float64."""
    g, u = np.asarray(g, dtype=np.float64), np.asarray(u, dtype=np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def gate_backward(g, u, dh):
    """((dg, |terms|), (du, |terms|)) in float64; |terms| bounds the magnitude of the
    products and sums that form each value (dg's slope 1 + g (1 - sigmoid) cancels)."""
    g, u, dh = (np.asarray(v, dtype=np.float64) for v in (g, u, dh))
    with np.errstate(over="ignore"):
        sg = 1.0 / (1.0 + np.exp(-g))
    dg = dh * u * sg * (1.0 + g * (1.0 - sg))
    du = dh * g * sg
    return (dg, np.abs(dh * u) * sg * (1.0 + np.abs(g) * (1.0 - sg))), (du, np.abs(du))


def decode_rows(q, s):
    """RN32(decode(code) * scale) of 1x128 codes q [R][K] with scales s [K/128][R]."""
    v = e4m3.decode(q).astype(np.float32)
    return v * np.repeat(np.asarray(s, np.float32).T, 128, axis=1)[:, :q.shape[1]]


def exp_error(x):
    """Relative error allowed to sigmoid(x) and to products with it in FP32: a few roundings
    (2^-21) and the exponential's argument reduction, whose absolute error in the
    exponent is |x| 2^-24 times a small factor."""
    return 2.0 ** -20 + np.abs(np.asarray(x, dtype=np.float64)) * 2.0 ** -23


def check_quantized(q, s, v, err, what):
    """Whether codes q [R][K] and scales s [K/128][R] (FP32) are a 1x128
    quantization of values within err of v: each scale within its group's largest err / 448
    and a float32 rounding, each decoded value within half an E4M3 step at its scale."""
    v, err = np.asarray(v, dtype=np.float64), np.broadcast_to(err, np.shape(v))
    R, K = v.shape
    if v.size == 0:
        return
    pad = -(-K // 128) * 128 - K
    groups = np.pad(np.abs(v), ((0, 0), (0, pad))).reshape(R, -1, 128)
    slack = np.pad(err, ((0, 0), (0, pad))).reshape(R, -1, 128).max(axis=2)
    want = groups.max(axis=2) / 448.0
    got = np.asarray(s, dtype=np.float64).T
    bad = np.argwhere(np.abs(got - want) > slack / 448.0 * (1 + 2.0 ** -20) + want * 2.0 ** -23 + 2.0 ** -149)
    assert bad.size == 0, f"{what}: {len(bad)} scales off, first {bad[:3].tolist()}"
    sc = np.repeat(got, 128, axis=1)[:, :K]
    value = e4m3.decode(q).astype(np.float64) * sc
    half = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * sc)
    bad = np.argwhere(np.abs(value - v) > half * (1 + 2.0 ** -8) + 2 * err + 2.0 ** -140)
    assert bad.size == 0, f"{what}: {len(bad)} codes off, first {bad[:3].tolist()}"


def finite_difference(f, x, at, step=1e-6):
    """Central difference of the scalar f at x along every index of `at`."""
    out = []
    for i in at:
        hi, lo = np.array(x, dtype=np.float64), np.array(x, dtype=np.float64)
        hi[i] += step
        lo[i] -= step
        out.append((f(hi) - f(lo)) / (2 * step))
    return np.array(out)

