"""Attention over a paged 8-bit key/value cache, from its definitions (test infrastructure only).

Plain loops over requests, pages and heads in float64: the pages, slots and
positions of a step, rotary positions, the quantization of new tokens into
pages under powers of two, and causal attention over the pages.  Nothing here
is shared with the HIP library.
"""

import numpy as np

from . import e4m3


def assign(have, add, table, free_pages, n_free, page, T):
    """(table, lens, cu, positions, slots, left) of a step; the arguments are not changed."""
    table = np.array(table)
    B, width = table.shape
    n = min(max(int(n_free), 0), len(free_pages))
    lens, cu = np.zeros(B, np.int64), np.zeros(B + 1, np.int64)
    positions, slots = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    row, wanted, taken = 0, 0, 0
    for b in range(B):
        h, a = max(int(have[b]), 0), max(int(add[b]), 0)
        a = min(a, T - row)
        held, need = -(-h // page), -(-(h + a) // page) - -(-h // page)
        fits = held + need <= width
        if fits:
            wanted += need
        given = fits and (need == 0 or wanted <= n)
        if given:
            for e in range(need):
                table[b, held + e] = free_pages[n - 1 - (wanted - need + e)]
            if need:
                taken = wanted
        lens[b] = h + a if given else h
        for i in range(a):
            positions[row + i] = h + i
            if given and table[b, (h + i) // page] >= 0:
                slots[row + i] = int(table[b, (h + i) // page]) * page + (h + i) % page
        row += a
        cu[b + 1] = row
    return table, lens, cu, positions, slots, np.array([n - taken, max(0, wanted - n)])


def release(done, lens, table, free_pages, n_free, page):
    """(lens, free_pages, left) after the done requests' pages went back."""
    free = list(np.array(free_pages))
    at = min(max(int(n_free), 0), len(free))
    out = np.maximum(np.array(lens), 0)
    for b in range(len(done)):
        if done[b]:
            for e in range(min(-(-int(out[b]) // page), table.shape[1])):
                if at < len(free):
                    free[at] = table[b][e]
                    at += 1
            out[b] = 0
    return out, np.array(free), at


def rope(x, positions, freqs, interleaved=False, scale=1.0, inverse=False):
    """x [T][H][D] with its first 2 len(freqs) channels turned, float64; rows with a negative position are zero."""
    x = np.asarray(x, np.float64)
    freqs = np.asarray(freqs, np.float64)
    half = len(freqs)
    out = np.zeros_like(x)
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        out[t] = x[t]
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            angle = float(pos) * freqs[i] * (-1.0 if inverse else 1.0)
            c, s = np.cos(angle) * scale, np.sin(angle) * scale
            out[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            out[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return out


def page_scale(amax):
    """The least power of two s >= 2^-126 with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    s = 2.0 ** -126
    while 448.0 * s < amax:
        s *= 2.0
    return s


def append(x, slots, codes, scale, page):
    """New rows x [T][H][D] into codes [n][H][page][D] and scale [n][H] (copies are returned): page after page."""
    x = np.asarray(x, np.float64)
    codes, scale = np.array(codes), np.array(scale, np.float64)
    n, H = scale.shape
    rows = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < n * page:
            rows.setdefault(int(slot) // page, []).append((int(slot) % page, t))
    for at, got in rows.items():
        first = min(o for o, _ in got)
        for h in range(H):
            s = page_scale(max(np.max(np.abs(x[t, h])) for _, t in got))
            if first > 0:
                was = scale[at, h]
                s = max(s, was)
                if s > was:
                    codes[at, h, :first] = e4m3.encode((e4m3.decode(codes[at, h, :first]) * (was / s)).astype(np.float32))
            for o, t in got:
                codes[at, h, o] = e4m3.encode((x[t, h] / (s if s > 0 else 1.0)).astype(np.float32))
            scale[at, h] = s
    return codes, scale


def values(codes, scale, table, length, page, h, turned=False):
    """The first `length` tokens [length][D] of a head of a request, and which of them are seen (their page exists)."""
    n = codes.shape[0]
    D = codes.shape[2] if turned else codes.shape[3]
    out, seen = np.zeros((length, D)), np.zeros(length, bool)
    for e in range(-(-length // page)):
        at = int(table[e])
        m = min(page, length - e * page)
        if 0 <= at < n:
            tile = codes[at, h].T if turned else codes[at, h]
            out[e * page: e * page + m] = e4m3.decode(tile[:m]) * float(scale[at, h])
            seen[e * page: e * page + m] = True
    return out, seen


def attention(q, k_cache, k_scale, v_cache, v_scale, table, cu, lens, scale):
    """(out [T][Hq][D], lse [T][Hq], size [T][Hq][D] = sum_j p_j |v_j|, score [T][Hq] = the largest
    scale * sum_d |q_d k_d|); rows of no request are 0."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    _, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    size, score = np.zeros(q.shape), np.zeros((T, Hq))
    for b in range(len(lens)):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        n = int(cu[b + 1] - cu[b])
        for h in range(Hkv):
            k, seen = values(k_cache, k_scale, table[b], length, page, h)
            v, _ = values(v_cache, v_scale, table[b], length, page, h, turned=True)
            for i in range(n):
                t = int(cu[b]) + i
                m = max(0, min(length - n + i + 1, length))
                live = seen[:m]
                if not live.any():
                    continue
                kk, vv = k[:m][live], v[:m][live]
                for j in range(h * G, (h + 1) * G):
                    x = scale * (kk @ q[t, j])
                    top = x.max()
                    e = np.exp(x - top)
                    p = e / e.sum()
                    out[t, j], lse[t, j] = p @ vv, top + np.log(e.sum())
                    size[t, j], score[t, j] = p @ np.abs(vv), scale * (np.abs(kk) @ np.abs(q[t, j])).max()
    return out, lse, size, score


def seen(q, k_cache, k_scale, v_scale, table, cu, lens, scale):
    """What an error of attention is measured by: (keys [T] that a row sees, p_max [T][Hq], the largest of its
    probabilities, top [T][Hq], the largest value scale of the pages of which it sees a token); 0 where it sees nothing."""
    q = np.asarray(q, np.float64)
    T, Hq, _ = q.shape
    n, Hkv, page, _ = k_cache.shape
    G = Hq // Hkv
    keys, p_max, top = np.zeros(T, np.int64), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(lens)):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        new = int(cu[b + 1] - cu[b])
        for h in range(Hkv):
            k, live = values(k_cache, k_scale, table[b], length, page, h)
            s = np.zeros(length)
            for j in np.nonzero(live)[0]:
                s[j] = float(v_scale[table[b][j // page], h])
            for i in range(new):
                t, m = int(cu[b]) + i, max(0, length - new + i + 1)
                if not live[:m].any():
                    continue
                keys[t] = live[:m].sum()
                x = scale * (k[:m][live[:m]] @ q[t, h * G: (h + 1) * G].T)
                p_max[t, h * G: (h + 1) * G] = 1.0 / np.exp(x - x.max(0)).sum(0)
                top[t, h * G: (h + 1) * G] = s[:m][live[:m]].max()
    return keys, p_max, top
