"""GPU parity of the paged 8-bit key/value cache's operators against the CPU oracle.

Pages, slots, positions, scales and codes must be equal; turned queries and keys
and attention stay within bounds derived from their roundings."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import e4m3, kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 2.0 ** -24                 # one FP32 rounding, relative


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def ints(a):
    return dev(np.asarray(a, np.int32))


def host(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def held(err, lim, what):
    bad = np.argwhere(~(np.abs(err) <= lim))
    assert bad.size == 0, f"{what}: {len(bad)} outside, first {bad[:3].tolist()}"


# ---------------------------------------------------------------------------
# pages

def pages_case(rng, B, most_have, most_add, page, width, spare):
    have = rng.integers(0, most_have + 1, B)
    add = rng.integers(0, most_add + 1, B)
    if B > 3:
        add[rng.integers(B)] = 0
        have[rng.integers(B)] = 0
        have[rng.integers(B)] = page * 2 if most_have >= 2 * page else 0
        add[-1] = 0
    have = np.minimum(have, width * page)
    ids = rng.permutation(B * width + 50)
    table = ids[:B * width].reshape(B, width).copy()
    for b in range(B):
        table[b, -(-have[b] // page):] = -7
    free = np.concatenate([ids[B * width:], np.arange(20)])
    return have, add, table, free, spare


@pytest.mark.parametrize("B,most_have,most_add,page,width,n_free,pad", [
    (1, 0, 1, 16, 1, 1, 0), (1, 40, 100, 64, 4, 50, 3), (5, 100, 3, 16, 8, 50, 0), (255, 90, 1, 32, 4, 50, 7), (256, 90, 1, 16, 8, 40, 0),
    (257, 300, 2, 64, 6, 50, 1), (600, 500, 40, 256, 3, 50, 5), (1000, 64, 1, 64, 2, 50, 1100), (30, 300, 300, 64, 9, 50, -500),
    (7, 400, 200, 128, 4, 2, 2), (9, 400, 2000, 16, 100, 50, 0), (300, 10, 0, 16, 1, 10, 5), (4, 33, 9, 16, 0, 10, 1)])
def test_assign(B, most_have, most_add, page, width, n_free, pad):
    rng = np.random.default_rng(B * 1000 + page)
    have, add, table, free, n = pages_case(rng, B, most_have, most_add, page, width, n_free)
    T = max(0, int(add.sum()) + pad)
    t = ints(table).reshape(B, width)
    got = fp8.kv_assign_pages(ints(have), ints(add), t, ints(free), ints([n]), page, T)
    want = kv.assign(have, add, table, free, n, page, T)
    for name, g, w in zip(("table", "lens", "cu", "positions", "slots", "left"), (t,) + got, want):
        assert np.array_equal(host(g), w), (name, host(g)[:20], w[:20])


def test_assign_odd_values():
    """Negative lengths, counts outside the list, empty batches."""
    for have, add, n in (([-5, 3], [2, -1], 4), ([0, 0], [2, 2], -3), ([0, 0], [2, 20], 100), ([2 ** 31 - 1, 5], [2 ** 31 - 1, 2 ** 31 - 1], 4)):
        table = np.zeros((2, 2), np.int64)
        t = ints(table)
        got = fp8.kv_assign_pages(ints(have), ints(add), t, ints([4, 5, 6, 7]), ints([n]), 16, 10)
        want = kv.assign(have, add, table, [4, 5, 6, 7], n, 16, 10)
        want = (want[0], want[1], want[2], np.minimum(want[3], 2 ** 31 - 1)) + want[4:]
        for g, w in zip((t,) + got, want):
            assert np.array_equal(host(g), w), (have, add, host(g), w)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    lens, cu, pos, slots, left = fp8.kv_assign_pages(none, none, torch.empty(0, 4, dtype=torch.int32, device=DEV), ints([1, 2]), ints([2]), 16, 3)
    assert cu.tolist() == [0] and pos.tolist() == [-1] * 3 and slots.tolist() == [-1] * 3 and left.tolist() == [2, 0]


@pytest.mark.parametrize("B,width,page,most,F,n_free", [
    (1, 1, 16, 16, 10, 0), (6, 5, 16, 90, 40, 3), (300, 9, 64, 500, 4000, 100), (257, 3, 256, 900, 100, 90), (1000, 8, 32, 256, 9000, 0),
    (50, 100, 16, 1600, 6000, 17), (3, 0, 16, 20, 5, 2)])
def test_release(B, width, page, most, F, n_free):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, most + 1, B)
    done = (rng.random(B) < 0.4) * rng.integers(1, 5, B)
    table = rng.integers(0, 10000, (B, width))
    free = rng.integers(0, 10000, F)
    f = ints(free)
    lens_out, left = fp8.kv_release_pages(ints(done), ints(lens), ints(table).reshape(B, width), f, ints([n_free]), page)
    want = kv.release(done, lens, table, free, n_free, page)
    assert np.array_equal(host(lens_out), want[0]) and np.array_equal(host(f), want[1]) and left.tolist() == [want[2]]


# ---------------------------------------------------------------------------
# rotary positions

@pytest.mark.parametrize("T,Hq,Hkv,D,rot,far", [
    (1, 1, 1, 64, 64, 10), (3, 5, 2, 128, 128, 2 ** 31 - 1), (7, 8, 1, 80, 80, 1000), (65, 3, 3, 192, 64, 100000), (130, 16, 4, 64, 32, 50),
    (5, 40, 8, 256, 256, 5000), (9, 2, 0, 96, 16, 77), (1030, 6, 2, 128, 48, 32768), (4, 1, 1, 8 * 128, 256, 9), (2, 300, 3, 64, 64, 100)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, Hq, Hkv, D, rot, far, bf16, interleaved):
    rng = np.random.default_rng(T + D)
    dt = torch.bfloat16 if bf16 else torch.float32
    freqs = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    pos = rng.integers(0, far, T)
    pos[-1] = far - 1
    if T > 4:
        pos[1] = pos[3] = -1                                   # rows of no request
    base = dev(rng.standard_normal((T, Hq + Hkv + 3, D)).astype(np.float32), dt)
    q, k = base[:, :Hq], base[:, Hq + 1: Hq + 1 + Hkv] if Hkv else None
    inverse, scale = bool(T % 2), 1.0 + 0.25 * (D % 3)
    qo, ko = torch.full((T, Hq, D), 7.0, dtype=dt, device=DEV), torch.full((T, Hkv + 2, D), 7.0, dtype=dt, device=DEV)
    out = fp8.rope(q, k, ints(pos), dev(freqs), interleaved, scale, inverse, q_out=qo, k_out=ko[:, 1: 1 + Hkv] if Hkv else None)
    for x, y in ((q, out[0]),) + (((k, out[1]),) if Hkv else ()):
        x, y = host(x).astype(np.float64), host(y)
        want = kv.rope(x, pos, freqs, interleaved, scale, inverse)
        dead = pos < 0
        assert np.all(y[dead] == 7.0)
        a = np.abs(x[..., :rot])
        a = a[..., 0::2] + a[..., 1::2] if interleaved else a[..., :rot // 2] + a[..., rot // 2:]
        size = np.abs(x)
        size[..., :rot] = np.repeat(a, 2, -1) if interleaved else np.tile(a, 2)
        # the turn's fraction in FP32 (half a turn at the most, pi 2^-25 in the angle), sine and cosine within two roundings,
        # their product with the scale, two products and a sum
        lim = scale * size * (np.pi * 2.0 ** -24 + 6 * EPS) + (2.0 ** -8 if bf16 else EPS) * np.abs(want)
        held((y - want)[~dead], lim[~dead], "rope")
        assert np.array_equal(y[~dead][..., rot:], x[~dead][..., rot:].astype(np.float32))
    assert torch.all(ko[:, :1] == 7.0) and torch.all(ko[:, 1 + Hkv:] == 7.0)


def test_rope_in_place_and_back():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(33, 12, 128, generator=g, device=DEV)
    freqs, scale = fp8.rope_frequencies(128, factor=4.0, device=DEV)
    pos = ints(np.arange(33) * 4000)
    for interleaved in (False, True):
        apart = fp8.rope(x[:, :8], x[:, 8:], pos, freqs, interleaved, scale)
        y = x.clone()
        fp8.rope(y[:, :8], y[:, 8:], pos, freqs, interleaved, scale, q_out=y[:, :8], k_out=y[:, 8:])
        assert torch.equal(y, torch.cat(apart, 1))
        fp8.rope(y[:, :8], y[:, 8:], pos, freqs, interleaved, 1.0 / scale, True, q_out=y[:, :8], k_out=y[:, 8:])
        assert torch.allclose(y, x, atol=1e-5)


# ---------------------------------------------------------------------------
# the cache

def random_cache(rng, n, H, page, D, special=True):
    k = rng.integers(0, 256, (n, H, page, D)).astype(np.uint8)
    v = rng.integers(0, 256, (n, H, D, page)).astype(np.uint8)
    for c in (k, v):
        if not special:
            c[(c & 0x7F) == 0x7F] = 0x30
    return k, v


def run_append(rng, T, slots, H, D, page, n, bf16, grow, scales=None, strided=False):
    x = rng.standard_normal((T, 2 * H + (1 if strided else 0), D)) * grow
    x = np.clip(x, -3e38, 3e38).astype(np.float32)                                # inputs are finite
    x[rng.random((T, 2 * H + strided)) < 0.1] = 0.0
    if T > 2:
        x[1] *= 2.0 ** -9
        x[2, :, ::3] *= 2.0 ** -12
    t = dev(x, torch.bfloat16 if bf16 else torch.float32)
    x = host(t)
    kc, vc = random_cache(rng, n, H, page, D, special=False)
    ks, vs = (2.0 ** rng.integers(-9, 3, (n, H)) if scales is None else np.full((n, H), scales) for _ in range(2))
    gpu = [dev(kc), dev(ks.astype(np.float32)), dev(vc), dev(vs.astype(np.float32))]
    k, v = (t[:, :H], t[:, H: 2 * H]) if strided else (t[:, :H].contiguous(), t[:, H: 2 * H].contiguous())
    fp8.fp8_kv_append(k, v, ints(slots), *gpu)
    wk, wks = kv.append(x[:, :H], slots, kc, ks, page)
    wv, wvs = kv.append(x[:, H: 2 * H], slots, vc.transpose(0, 1, 3, 2), vs, page)
    for name, g, w in zip(("keys' scales", "values' scales", "keys", "values"), (gpu[1], gpu[3], gpu[0], gpu[2]), (wks, wvs, wk, wv.transpose(0, 1, 3, 2))):
        g = host(g)
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:4].tolist(), g[g != w][:4], w[g != w][:4])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,H,bf16,strided", [(64, 3, True, False), (128, 2, False, True), (192, 1, True, True), (256, 2, True, False)])
def test_append(page, D, H, bf16, strided):
    """Runs that start a page, fill one up, cross into the next, single tokens, skipped rows."""
    rng = np.random.default_rng(page + D)
    runs = [(0, 1), (page - 1, 2), (5, page), (0, 2 * page + 3), (page - 3, 3), (1, 1), (page // 2, 7)]      # offset, tokens
    ids, slots = list(rng.permutation(30)), []
    for off, count in runs:
        at, left = ids.pop(), count
        while left > 0:
            m = min(left, page - off)
            slots += [at * page + off + i for i in range(m)]
            left, off = left - m, 0
            at = ids.pop() if left else at
        slots.append([-1, 30 * page, 2 ** 31 - 1][len(slots) % 3])
    for grow in (1.0, 2.0 ** -8, 300.0):
        run_append(rng, len(slots), slots, H, D, page, 30, bf16, grow, strided=strided)


def test_append_extremes():
    """Scales at FP32's ends, pages of zeros, values at the code's largest."""
    rng = np.random.default_rng(3)
    for grow, scales in ((1e38, None), (1e-38, 2.0 ** -126), (1e-41, 2.0 ** -126), (1.0, 0.0), (1e30, 2.0 ** -126), (0.0, 0.0), (1e-30, 2.0 ** 100)):
        run_append(rng, 9, [0, 1, 2, 20, 21, 22, 40, 41, 48], 2, 64, 16, 4, False, grow, scales)
    for top in (448.0, 447.0, 449.0, 1.75, 1.7500001):
        x = torch.full((1, 1, 64), top, device=DEV)
        cache = fp8.kv_cache(1, 1, 16, 64, DEV)
        fp8.fp8_kv_append(x, -x, ints([0]), *cache)
        assert cache[1].item() == cache[3].item() == kv.page_scale(float(np.float32(top)))


def test_append_token_by_token_keeps_what_one_call_gives():
    """A page filled a token at a time, in any growth of its scale, holds what one call writes, but for codes that had become subnormal."""
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((64, 2, 64)) * 2.0 ** rng.integers(-3, 4, (64, 1, 1))).astype(np.float32)
    t = dev(x)
    one, many = fp8.kv_cache(2, 2, 64, 64, DEV), fp8.kv_cache(2, 2, 64, 64, DEV)
    fp8.fp8_kv_append(t, t, ints(64 + np.arange(64)), *one)
    for i in range(64):
        fp8.fp8_kv_append(t[i:i + 1], t[i:i + 1], ints([64 + i]), *many)
    assert torch.equal(one[1], many[1]) and torch.equal(one[3], many[3])
    for a, b in ((one[0], many[0]), (one[2], many[2])):
        va, vb = (e4m3.decode(host(c)) for c in (a, b))
        assert np.max(np.abs(va - vb)) <= 2.0 ** -9            # one subnormal step: two roundings, of half a step each
        assert np.array_equal(va[np.abs(va) > 2.0 ** -5], vb[np.abs(va) > 2.0 ** -5])


# ---------------------------------------------------------------------------
# attention

def attention_case(rng, held_, new, Hq, Hkv, D, page, pad=0, special=True, width=None, scales=None, loud=1.0):
    lens = [h + n for h, n in zip(held_, new)]
    counts = [-(-n // page) for n in lens]
    width = max(max(counts), 1) if width is None else width
    n_pages = sum(counts) + 3
    ids = rng.permutation(n_pages)
    table, at = rng.integers(-5, n_pages + 5, (len(lens), width)), 0
    k, v = random_cache(rng, n_pages, Hkv, page, D, special)
    ks, vs = ((2.0 ** rng.integers(-9, -6, (n_pages, Hkv))).astype(np.float32) if scales is None else scales(rng, (n_pages, Hkv)) for _ in range(2))
    finite = (np.arange(256) & 0x7F) != 0x7F
    unused = np.ones(n_pages, bool)
    for b, c in enumerate(counts):
        c = min(c, width)
        table[b, :c] = ids[at: at + c]
        unused[ids[at: at + c]] = False
        for e in range(c):                                     # codes of tokens are numbers, the rest of a page is anything
            m = min(page, lens[b] - e * page)
            for tile in (k[table[b, e], :, :m], v[table[b, e], :, :, :m]):
                tile[~finite[tile]] = 0x38
        at += c
    if special:
        ks[unused], vs[unused] = np.nan, np.inf
    T = sum(new) + pad
    q = torch.from_numpy((rng.standard_normal((T, Hq, D)) * loud).astype(np.float32)).bfloat16()
    cu = np.concatenate([[0], np.cumsum(new)])
    return q, k, ks, v, vs, table, cu, np.array(lens)


def attention_check(case, scale=None, **more):
    q, k, ks, v, vs, table, cu, lens = case
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    gq = q.to(DEV)
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 9.0, device=DEV)
    gpu = (dev(k), dev(ks), dev(v), dev(vs), ints(table).reshape(table.shape), ints(cu), ints(lens))
    fp8.fp8_kv_attention(gq, *gpu, scale, out, lse, **more)
    again = fp8.fp8_kv_attention(gq, *gpu, scale)
    used = int(cu[-1])
    assert torch.equal(out[:used], again[:used])
    o, l = host(out), host(lse)
    assert np.all(o[used:] == 9.0) and np.all(l[used:] == 9.0)
    want, wlse, size, score = kv.attention(q.float().numpy(), k, ks, v, vs, table, cu, lens, scale)
    o, l, want, wlse, size, score = (a[:used] for a in (o, l, want, wlse, size, score))
    n = int(lens.max()) if len(lens) else 0
    # a score: D products summed in FP32, two factors; its exponential: the scaled argument's rounding and the exponential's own
    x = (D + 8) * EPS * score + 4 * EPS
    # p in FP16 (half a step 2^-11), sums over the tokens in FP32, the normalisation and the joining factors
    p = 2.0 ** -11 + 4 * x + (n + 64) * EPS
    vmax = float(np.nanmax(np.where(np.isfinite(vs), np.abs(vs), 0))) * 448.0
    lim = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * p[..., None] * size + 2.0 ** -50 * vmax
    held(o - want, lim, "out")
    empty = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(l), empty) and np.all(o[empty] == 0)
    held((l - wlse)[~empty], (2 * x + (n + 64) * EPS + 8 * EPS * np.abs(wlse))[~empty], "lse")
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode(D, page):
    """One new token each: lengths at the ends of pages and tiles, requests without a token, in a padded batch."""
    rng = np.random.default_rng(D + page)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 255, 256, 257, 300, 511, 700, 1025]
    new = [1] * len(lens)
    new[3] = new[7] = 0
    attention_check(attention_case(rng, [n - a for n, a in zip(lens, new)], new, 4, 2, D, page, pad=2))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (7, 1), (12, 4), (8, 8), (16, 1), (34, 2), (71, 1), (40, 8)])
def test_head_layouts(Hq, Hkv):
    rng = np.random.default_rng(Hq)
    attention_check(attention_case(rng, [0, 33, 500, 0, 90], [1, 2, 1, 5, 3], Hq, Hkv, 64, 32, pad=1))


@pytest.mark.parametrize("D,page,Hq,Hkv,held_,new", [
    (128, 64, 8, 2, [0], [200]), (64, 16, 4, 4, [100, 0, 7], [65, 64, 1]), (128, 128, 16, 1, [300, 0], [17, 130]),
    (256, 64, 2, 2, [64, 63], [64, 65]), (192, 32, 6, 2, [10, 500, 0, 3], [40, 1, 0, 33]), (128, 16, 5, 1, [1000], [3]),
    (64, 256, 8, 1, [255, 256, 257], [2, 2, 2]), (128, 64, 32, 4, [0, 4100], [70, 9])])
def test_chunks(D, page, Hq, Hkv, held_, new):
    rng = np.random.default_rng(sum(new))
    attention_check(attention_case(rng, held_, new, Hq, Hkv, D, page, pad=5))


@pytest.mark.parametrize("held_,new,Hq,Hkv", [([5000], [1], 4, 1), ([9000, 10, 0, 2500], [1, 1, 1, 1], 8, 2), ([4097, 6000], [3, 2], 8, 1),
                                              ([70, 12000], [40, 2], 4, 4)])
def test_long_axis(held_, new, Hq, Hkv):
    """Keys split over workgroups and joined, short requests beside long ones."""
    rng = np.random.default_rng(held_[0])
    attention_check(attention_case(rng, held_, new, Hq, Hkv, 128, 64, pad=1))


@pytest.mark.parametrize("D,page", [(64, 128), (128, 16), (192, 64), (256, 32)])
def test_long_axis_of_many_rows(D, page):
    """Many rows over keys that are split: their parts joined row by row, beside requests that are not split."""
    rng = np.random.default_rng(D)
    attention_check(attention_case(rng, [2500, 0, 1200, 30], [45, 70, 0, 133], 3, 1, D, page, pad=2))


def test_rows_that_see_nothing():
    """Requests shorter than their new rows (refused ones), empty ones, and a batch of nothing else."""
    rng = np.random.default_rng(8)
    q, k, ks, v, vs, table, cu, lens = attention_case(rng, [0, 24, 3, 38], [4, 6, 1, 2], 6, 2, 128, 16, pad=1)
    lens = np.array([2, 0, 4, 1])
    attention_check((q, k, ks, v, vs, table, cu, lens))
    attention_check((q, k, ks, v, vs, table, cu, np.zeros(4, int)))
    attention_check((q, k, ks, v, vs, table[:, :1], cu, np.array([2, 30, 4, 40])))       # tokens past the table's last entry
    attention_check((q, k, ks, v, vs, table[:, :0], cu, np.array([2, 30, 4, 40])))


def test_pages_that_do_not_exist():
    rng = np.random.default_rng(9)
    q, k, ks, v, vs, table, cu, lens = attention_case(rng, [300, 40, 600], [1, 2, 3], 4, 2, 64, 16, pad=0)
    table[0, 3], table[0, 18], table[1, :] = -1, k.shape[0], 2 ** 31 - 1
    table[2, 0:9] = -2 ** 31
    attention_check((q, k, ks, v, vs, table, cu, lens))


@pytest.mark.parametrize("page", [16, 64])
def test_scales_far_apart(page):
    """Any FP32 scales: neighbouring pages' far apart, zeros among them."""
    rng = np.random.default_rng(10)
    for lo, hi in ((-30, 30), (-14, -4)):
        def scales(r, shape):
            s = (2.0 ** r.uniform(lo, hi, shape)).astype(np.float32)
            s[r.random(shape) < 0.2] = 0.0
            return s
        case = attention_case(rng, [500, 77, 40], [1, 1, 6], 4, 2, 64, page, scales=scales, special=False)
        case[2][...] = np.where(case[2] > 0, 2.0 ** -7, case[2])          # keys of ordinary size
        attention_check(case)


def test_loud_scores_and_flat_ones():
    rng = np.random.default_rng(11)
    attention_check(attention_case(rng, [200, 64], [1, 3], 4, 2, 128, 64, loud=30.0))
    attention_check(attention_case(rng, [200, 64], [1, 3], 4, 2, 128, 64), scale=0.0)
    case = attention_case(rng, [1000], [2], 4, 2, 64, 16, loud=0.01)
    attention_check(case)


def test_strided_queries_and_workspace():
    rng = np.random.default_rng(12)
    q, k, ks, v, vs, table, cu, lens = attention_case(rng, [2000, 30], [2, 5], 8, 2, 128, 64)
    wide = torch.zeros(q.shape[0], 12, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10] = q.to(DEV)
    gpu = (dev(k), dev(ks), dev(v), dev(vs), ints(table), ints(cu), ints(lens))
    need = fp8.fp8_kv_attention_workspace(q.shape[0], 2, 8, 2, 128, 64, table.shape[1])
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    a = fp8.fp8_kv_attention(wide[:, 2:10], *gpu, workspace=ws)
    b = fp8.fp8_kv_attention(q.to(DEV), *gpu)
    assert torch.equal(a, b) and torch.all(ws[need:] == 255)
    with pytest.raises(fp8.Fp8fgError):
        fp8.fp8_kv_attention(q.to(DEV), *gpu, workspace=ws[:need - 64])
    with pytest.raises(ValueError):
        fp8.fp8_kv_attention(q.to(DEV).transpose(0, 1), *gpu)


# ---------------------------------------------------------------------------
# together

class Server:
    """A few requests served by the operators, and the same by the oracle: the cache's contents are compared at every step."""

    def __init__(self, B, Hq, Hkv, D, page, width, n_pages, T, seed):
        self.Hq, self.Hkv, self.D, self.page, self.T = Hq, Hkv, D, page, T
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.have = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.add = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.arange(n_pages, dtype=torch.int32, device=DEV)
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=DEV)
        self.cache = fp8.kv_cache(n_pages, Hkv, page, D, DEV)
        self.freqs, self.scale = fp8.rope_frequencies(D, device=DEV)
        self.x = torch.empty(T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)

    def feed(self, add):
        self.add.copy_(ints(add))
        self.x.copy_(torch.randn(self.x.shape, generator=self.g, device=DEV))

    def step(self):
        lens, cu, pos, slots, left = fp8.kv_assign_pages(self.have, self.add, self.table, self.free, self.n_free, self.page, self.T)
        q, k = fp8.rope(self.x[:, :self.Hq], self.x[:, self.Hq:self.Hq + self.Hkv], pos, self.freqs, scale=self.scale)
        fp8.fp8_kv_append(k, self.x[:, self.Hq + self.Hkv:], slots, *self.cache)
        out = fp8.fp8_kv_attention(q, *self.cache, self.table, cu, lens)
        self.have.copy_(lens)
        self.n_free.copy_(left[:1])
        return lens, cu, pos, slots, q, out


def test_requests_come_and_go():
    B, T, page = 5, 40, 16
    s = Server(B, 8, 2, 64, page, 8, 16, T, 1)
    rng = np.random.default_rng(1)
    keys = [np.zeros((0, 2, 64)) for _ in range(B)]
    vals = [np.zeros((0, 2, 64)) for _ in range(B)]
    for step in range(14):
        add = rng.integers(0, 9 if step % 4 == 0 else 3, B)
        before = host(s.have).copy()
        s.feed(add)
        lens, cu, pos, slots, q, out = s.step()
        x = host(s.x).astype(np.float64)
        lens, cu, pos = host(lens), host(cu), host(pos)
        assert len(set(host(s.table)[b, e] for b in range(B) for e in range(-(-lens[b] // page)))) == sum(-(-lens // page))
        k = kv.rope(x[:, 8:10], pos, host(s.freqs))
        for b in range(B):
            if lens[b] == before[b] + add[b]:
                keys[b] = np.concatenate([keys[b], k[cu[b]:cu[b + 1]]])
                vals[b] = np.concatenate([vals[b], x[cu[b]:cu[b + 1], 10:12]])
            assert len(keys[b]) == lens[b]
            for h in range(2):
                for c, sc, have, turned in ((s.cache[0], s.cache[1], keys[b], False), (s.cache[2], s.cache[3], vals[b], True)):
                    got, seen = kv.values(host(c), host(sc), host(s.table)[b], lens[b], page, h, turned)
                    assert seen.all()
                    # E4M3 twice at the most where a scale grew (half a step is 2^-4 of the value), the turned keys' rounding to
                    # BF16, and the code's smallest steps under scales of 2^-6 and less (|x| < 28)
                    lim = np.abs(have[:, h]) * (2.0 ** -4 + 2.0 ** -8 * 2) + 2.0 ** -6 * 2.0 ** -9
                    held(got - have[:, h], lim, (step, b))
        args = [host(t) for t in s.cache] + [host(s.table), cu, lens, 64 ** -0.5]
        want, _, size, _ = kv.attention(host(q), *args)
        live = slice(0, cu[-1])
        held(host(out)[live] - want[live], (2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size)[live], step)
        if step in (5, 9):                                     # two requests end
            done = np.zeros(B, int)
            done[[step % B, (step + 2) % B]] = 1
            lens, left = fp8.kv_release_pages(ints(done), s.have, s.table, s.free, s.n_free, page)
            s.have.copy_(lens)
            s.n_free.copy_(left)
            for b in np.nonzero(done)[0]:
                keys[b], vals[b] = keys[b][:0], vals[b][:0]


def test_a_step_captured_and_replayed():
    s, e = (Server(6, 8, 2, 128, 16, 30, 200, 12, 5) for _ in range(2))
    rng = np.random.default_rng(6)
    state = [t.clone() for t in (s.have, s.table, s.n_free, *s.cache)]
    s.feed(np.ones(6))
    s.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step()
    for t, was in zip((s.have, s.table, s.n_free, *s.cache), state):
        t.copy_(was)
    s.g.manual_seed(5)
    for step in range(12):
        add = rng.integers(0, 3, 6) if step else np.full(6, 2)
        s.feed(add)
        e.feed(add)
        graph.replay()
        mine = [t.clone() for t in got]
        torch.cuda.synchronize()
        want = e.step()
        used = int(want[1][-1])
        for n, (a, b) in enumerate(zip(mine, want)):
            assert torch.equal(a[:used] if n > 3 else a, b[:used] if n > 3 else b), (step, n)
        for a, b in zip(s.cache, e.cache):
            assert torch.equal(a, b)


def test_on_another_stream_and_two_at_once():
    """Calls on two streams at once, each with its own outputs and workspace."""
    rng = np.random.default_rng(13)
    cases = [attention_case(rng, [3000 + 500 * i, 40], [1, 3], 8, 2, 128, 64) for i in range(2)]
    gpu = [(c[0].to(DEV), dev(c[1]), dev(c[2]), dev(c[3]), dev(c[4]), ints(c[5]), ints(c[6]), ints(c[7])) for c in cases]
    want = [fp8.fp8_kv_attention(*c) for c in gpu]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(fp8.fp8_kv_attention(*gpu[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


@pytest.mark.parametrize("G,add,long", [(1, 1, 0), (3, 1, 3000), (2, 40, 0), (40, 2, 0)])
def test_many_requests(G, add, long):
    """More requests than a wave looks at together, most of them short, one long one among them: each kernel."""
    rng = np.random.default_rng(G)
    B = 270 if add == 1 else 262
    held_ = list(rng.integers(0, 40, B))
    new = [add if i % 5 else 0 for i in range(B)] if add == 1 else [1 + i % add if i % 7 else 0 for i in range(B)]
    if long:
        held_[200] = long
    attention_check(attention_case(rng, held_, new, G, 1, 64, 16, pad=3))


def test_only_long_tiles_split():
    """More row tiles than workgroups run at a time; the few of a long request are split, the others whole."""
    rng = np.random.default_rng(33)
    q, k, ks, v, vs, table, cu, lens = attention_case(rng, [0, 3500], [1200, 150], 64, 64, 64, 64)
    lse = torch.empty(q.shape[:2], device=DEV)
    out, _ = fp8.fp8_kv_attention(q.to(DEV), dev(k), dev(ks), dev(v), dev(vs), ints(table), ints(cu), ints(lens), lse=lse)
    for h in (0, 37, 63):
        part = [a[:, h: h + 1].copy() for a in (k, ks, v, vs)]
        one = (q[:, h: h + 1].contiguous(), *part, table, cu, lens)
        n, got = int(lens.max()), host(out[:, h: h + 1])
        full, flse, size, score = kv.attention(one[0].float().numpy(), *part, table, cu, lens, 64 ** -0.5)
        x = (64 + 8) * EPS * score + 4 * EPS
        p = 2.0 ** -11 + 4 * x + (n + 64) * EPS
        vmax = float(np.nanmax(np.where(np.isfinite(part[3]), np.abs(part[3]), 0))) * 448.0
        held(got - full, 2.0 ** -8 * np.abs(full) + (1 + 2.0 ** -8) * p[..., None] * size + 2.0 ** -50 * vmax, "out")
        held(host(lse[:, h: h + 1]) - flse, 2 * x + (n + 64) * EPS + 8 * EPS * np.abs(flse), "lse")


def test_list_across_chunks():
    """Requests in several chunks of 256, empty, short and split ones in each, replayed from a graph on other lengths."""
    rng = np.random.default_rng(21)
    B = 700
    cases = []
    for k in range(2):
        held_ = rng.integers(0, 30, B)
        held_[[3 + k, 300 + k, 650 + k]] = 2500 + 100 * k
        cases.append(attention_case(rng, list(held_), [int(i % 4 > 0) for i in range(B)], 2, 1, 64, 16, pad=5, width=170))
        attention_check(cases[-1])
    gpu = [(c[0].to(DEV), dev(c[1]), dev(c[2]), dev(c[3]), dev(c[4]), ints(c[5]), ints(c[6]), ints(c[7])) for c in cases]
    most = max(g[1].shape[0] for g in gpu)
    at = [torch.zeros((most, *x.shape[1:]) if 1 <= i <= 4 else x.shape, dtype=x.dtype, device=DEV) for i, x in enumerate(gpu[0])]

    def put(g):
        for a, x in zip(at, g):
            a[:x.shape[0]].copy_(x)

    put(gpu[0])
    out = torch.zeros_like(at[0])
    fp8.fp8_kv_attention(*at, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.fp8_kv_attention(*at, out=out)
    for k in (1, 0, 1, 0):
        put(gpu[k])
        graph.replay()
        torch.cuda.synchronize()
        used = int(gpu[k][6][-1])
        assert torch.equal(out[:used], fp8.fp8_kv_attention(*gpu[k])[:used])


def test_empty_problems():
    """No requests, no rows: what exists is written, nothing else."""
    none, free, n = ints([]), ints([5, 6, 7]), ints([3])
    table = ints([]).reshape(0, 4)
    lens, cu, positions, slots, left = fp8.kv_assign_pages(none, none, table, free, n, 16, 3)
    assert lens.numel() == 0 and cu.tolist() == [0] and positions.tolist() == slots.tolist() == [-1] * 3 and left.tolist() == [3, 0]
    table = ints([[-1, -1], [4, -1]])
    lens, cu, positions, slots, left = fp8.kv_assign_pages(ints([0, 9]), ints([2, 0]), table, free, n, 16, 0)
    assert lens.tolist() == [0, 9] and cu.tolist() == [0, 0, 0] and positions.numel() == slots.numel() == 0 and left.tolist() == [3, 0]
    assert table.tolist() == [[-1, -1], [4, -1]]
    lens, left = fp8.kv_release_pages(none, none, ints([]).reshape(0, 4), free, n, 16)
    assert lens.numel() == 0 and left.tolist() == [3] and free.tolist() == [5, 6, 7]
    cache = fp8.kv_cache(2, 1, 16, 64, DEV)
    x = torch.ones(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    assert fp8.rope(x, x, none, torch.ones(32, device=DEV))[0].shape == x.shape
    fp8.fp8_kv_append(x, x, none, *cache)
    assert all(int(t.count_nonzero()) == 0 for t in cache)
    assert fp8.fp8_kv_attention(x, *cache, ints([[0]]), ints([0, 0]), ints([7])).shape == x.shape
    out = torch.full((2, 1, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    fp8.fp8_kv_attention(out.clone(), *cache, ints([]).reshape(0, 1), ints([0]), none, out=out)
    assert bool((out == 3.0).all())


def test_most_requests():
    """65,536 requests of one token each through every call: the token sees itself alone, so that
    the output is its value as the cache holds it, and lse the one score."""
    B, page, D = 65536, 16, 64
    g = torch.Generator(device=DEV).manual_seed(17)
    free = torch.randperm(B, generator=g, device=DEV).int()
    have, add = torch.zeros(B, dtype=torch.int32, device=DEV), torch.ones(B, dtype=torch.int32, device=DEV)
    table = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    lens, cu, positions, slots, left = fp8.kv_assign_pages(have, add, table, free, ints([B]), page, B)
    assert torch.equal(table[:, 0], free.flip(0)) and torch.equal(slots, table[:, 0] * page) and left.tolist() == [0, 0]
    assert torch.equal(cu, torch.arange(B + 1, dtype=torch.int32, device=DEV)) and int(positions.abs().max()) == 0
    cache = fp8.kv_cache(B, 1, page, D, DEV)
    x = torch.randn(B, 3, D, generator=g, device=DEV).bfloat16()
    fp8.fp8_kv_append(x[:, 1:2], x[:, 2:], slots, *cache)
    lse = torch.empty(B, 1, device=DEV)
    out, _ = fp8.fp8_kv_attention(x[:, :1], *cache, table, cu, lens, lse=lse)
    at = table[:, 0].long()
    k = e4m3.decode(host(cache[0][at, 0, 0])) * host(cache[1][at]).astype(np.float64)
    v = e4m3.decode(host(cache[2][at, 0, :, 0])) * host(cache[3][at]).astype(np.float64)
    # p = 1 up to FP32 roundings and a power of two as the scale: values of four bits are BF16's own
    assert np.array_equal(host(out)[:, 0], v)
    score = D ** -0.5 * (host(x[:, 0]) * k).sum(1)
    size = D ** -0.5 * np.abs(host(x[:, 0]) * k).sum(1)
    # as in attention_check, with one token
    held(host(lse)[:, 0] - score, 2 * ((D + 8) * EPS * size + 4 * EPS) + 65 * EPS + 8 * EPS * np.abs(score), "lse")
    lens, left = fp8.kv_release_pages(add, lens, table, free, ints([0]), page)
    assert torch.equal(free, table[:, 0]) and int(lens.abs().max()) == 0 and left.tolist() == [B]


def test_offsets_past_32_bits():
    """Pages far into a cache of more than 4 GB: writes and reads land where the small cache's do."""
    H, page, D, n = 4, 256, 256, 17000
    g = torch.Generator(device=DEV).manual_seed(3)
    big = (torch.empty(n, H, page, D, dtype=torch.uint8, device=DEV), torch.empty(n, H, device=DEV),
           torch.empty(n, H, D, page, dtype=torch.uint8, device=DEV), torch.empty(n, H, device=DEV))
    small = fp8.kv_cache(4, H, page, D, DEV)
    ids = [16999, 1, 16500, 8191]
    T = 700
    x = torch.randn(T, 3 * H, D, generator=g, device=DEV).bfloat16()
    for cache, table in ((big, ids), (small, [0, 1, 2, 3])):
        slots = [table[i // page] * page + i % page for i in range(600)] + [table[3] * page + i for i in range(100)]
        fp8.fp8_kv_append(x[:, H:2 * H], x[:, 2 * H:], ints(slots), *cache)
    for a, b in zip(big, small):
        assert torch.equal(a[ids[:2]], b[:2])
    for cu, lens in (([0, 600, 700], [600, 100]), ([0, 1, 2], [600, 100])):
        out = []
        for cache, table in ((big, ids), (small, [0, 1, 2, 3])):
            tab = ints([table[:3], [table[3]] * 3])
            out.append(fp8.fp8_kv_attention(x[:cu[-1], :H], *cache, tab, ints(cu), ints(lens)))
        assert torch.equal(*out)


def test_two_graphs_with_one_workspace():
    """Two captured calls that share a workspace, replayed in turn."""
    rng = np.random.default_rng(14)
    cases = [attention_case(rng, h, n, 8, 2, 128, 64) for h, n in (([3000, 40], [1, 3]), ([20, 4500, 1000], [2, 1, 1]))]
    gpu = [(c[0].to(DEV), dev(c[1]), dev(c[2]), dev(c[3]), dev(c[4]), ints(c[5]), ints(c[6]), ints(c[7])) for c in cases]
    need = max(fp8.fp8_kv_attention_workspace(c[0].shape[0], len(c[7]), 8, 2, 128, 64, c[5].shape[1]) for c in cases)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = [fp8.fp8_kv_attention(*c) for c in gpu]
    graphs, got = [], []
    for c in gpu:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(fp8.fp8_kv_attention(*c, workspace=ws))
        graphs.append(g)
    for k in range(6):
        got[k % 2].zero_()
        graphs[k % 2].replay()
        ws.fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(got[k % 2], want[k % 2]), k
