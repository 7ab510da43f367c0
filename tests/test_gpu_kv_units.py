"""Attention over value scales that lie far apart: each row's error against the largest scale that the row itself sees.

|out - out*| <= (2^-11 + 2^-22 (D + 8) X + 2^-24 (n + 128)) sum_j p_j |v_j| + 2^-27 p_max n max(S, 2^-100) + 2^-100 before the rounding
to BF16, with n the keys that a row sees, X the largest scale * sum_d |q_d k_jd|, p_max the row's largest probability and S the largest
value scale of the pages of which it sees a token: half a step of FP16; four times a score's error, of D products' sum in FP32; the sums
over keys and parts; and 448 times half of FP16's smallest step, 2^-25, over the least that the largest probability is held as, 2^11."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import kv
from tests.test_gpu_kv import DEV, EPS, attention_case, dev, held, host, ints

pytestmark = pytest.mark.gpu

# Each kernel: 16, 32 and 128 query rows a workgroup, with and without keys that are split over workgroups (tables of more than 1024 tokens)
FORMS = [("16", 64, 2, 2, 30, 5), ("16 split", 128, 2, 1, 1502, 5), ("16, D = 256", 256, 4, 2, 30, 3), ("32", 64, 8, 2, 30, 6), ("32 split", 128, 6, 1, 1310, 5),
         ("128", 64, 2, 1, 40, 70), ("128 split", 128, 4, 2, 1502, 40), ("128, D = 192", 192, 1, 1, 20, 75), ("128, D = 256", 256, 2, 1, 90, 70)]
each_form = pytest.mark.parametrize("Hq,Hkv,D,old,new", [f[2:4] + f[1:2] + f[4:] for f in FORMS], ids=[f[0] for f in FORMS])


def on_gpu(case):
    q, k, ks, v, vs, table, cu, lens = case
    return q.to(DEV), dev(k), dev(ks.astype(np.float32)), dev(v), dev(vs.astype(np.float32)), ints(table).reshape(table.shape), ints(cu), ints(lens)


def bound_check(case):
    q, k, ks, v, vs, table, cu, lens = case
    T, Hq, D = q.shape
    scale, x = D ** -0.5, q.float().numpy()
    lse = torch.empty(T, Hq, device=DEV)
    out, _ = fp8.fp8_kv_attention(*on_gpu(case), lse=lse)
    want, wlse, size, score = kv.attention(x, k, ks, v, vs, table, cu, lens, scale)
    keys, p_max, top = kv.seen(x, k, ks, vs, table, cu, lens, scale)
    x = (D + 8) * EPS * score + 4 * EPS
    lim = (2.0 ** -11 + 4 * x + (keys[:, None] + 112) * EPS)[..., None] * size + (2.0 ** -27 * keys[:, None] * p_max * np.maximum(top, 2.0 ** -100))[..., None] + 2.0 ** -100
    held(host(out) - want, lim + 2.0 ** -8 * (np.abs(want) + lim), "out")
    held(host(lse) - wlse, 2 * x + (keys[:, None] + 64) * EPS + 8 * EPS * np.abs(wlse), "lse")
    return out


def spread(rng, old, new, Hq, Hkv, D, page, scale_of):
    """Two requests, the second without older tokens, whose e-th pages have the value scale scale_of(e, pages)."""
    case = list(attention_case(rng, [old, 0], [new, new], Hq, Hkv, D, page, special=False))
    table, lens, vs = case[5], case[7], case[4].astype(np.float64)
    case[2] = np.full(case[2].shape, 2.0 ** -8)                # keys of ordinary size
    vs[...] = 1.0
    for b, n in enumerate(lens):
        pages = -(-int(n) // page)
        for e in range(pages):
            vs[table[b, e]] = scale_of(e, pages)
    case[4] = vs
    return case


@pytest.mark.parametrize("far", [20, 40, 100])
@pytest.mark.parametrize("page", [16, 32])
@each_form
def test_later_pages_of_far_larger_scales(page, far, Hq, Hkv, D, old, new):
    """Tokens that do not see a request's last page, whose scale is 2^far times the others', as if it had the others'."""
    bound_check(spread(np.random.default_rng(D + far), old, new, Hq, Hkv, D, page, lambda e, pages: 2.0 ** (far - 8 if e == pages - 1 else -8)))


@pytest.mark.parametrize("step", [-20, 20, -5])
@each_form
def test_scales_that_rise_and_fall(step, Hq, Hkv, D, old, new):
    """Every page's scale 2^step times that of the page before, within 2^-90 .. 2^60."""
    bound_check(spread(np.random.default_rng(D + step), old, new, Hq, Hkv, D, 16, lambda e, pages: 2.0 ** np.clip((e - pages // 2) * step, -90, 60)))


@pytest.mark.parametrize("page", [16, 32])
@each_form
def test_pages_that_a_row_does_not_see_leave_its_bits(page, Hq, Hkv, D, old, new):
    """Codes and scales of a request's last page change; the outputs of the tokens before it do not."""
    rng = np.random.default_rng(D + page)
    case = spread(rng, old, new, Hq, Hkv, D, page, lambda e, pages: 2.0 ** (-8 + 3 * (e % 4)))
    q, k, ks, v, vs, table, cu, lens = case
    changed = [a.copy() for a in (k, ks, v, vs)]
    for b, n in enumerate(lens):
        at = table[b, -(-int(n) // page) - 1]
        changed[0][at], changed[2][at] = changed[0][at] ^ 0x80, changed[2][at] ^ 0x88
        changed[2][at][(changed[2][at] & 0x7F) == 0x7F] = 0x38
        changed[1][at], changed[3][at] = 0.37, 1.7e30
    outs = []
    for a, b, c, d in ((k, ks, v, vs), changed):
        lse = torch.empty(q.shape[:2], device=DEV)
        outs.append(fp8.fp8_kv_attention(*on_gpu((q, a, b, c, d, table, cu, lens)), lse=lse))
    rows = 0
    for b, n in enumerate(lens):
        before = (-(-int(n) // page) - 1) * page - (int(n) - new)           # the request's new tokens before its last page
        for i in range(max(0, before)):
            assert all(torch.equal(x[cu[b] + i], y[cu[b] + i]) for x, y in zip(*outs)), (b, i)
            rows += 1
    assert rows > 0


# value scale, largest code: values up to 3.2e38, and those of the smallest scales, which the bound's last terms cover
@pytest.mark.parametrize("top,code", [(2.0 ** 110, 0x7E), (2.0 ** 119, 0x7E), (2.0 ** 120, 0x77), (1.9 * 2.0 ** 126, 0x40), (1.9 * 2.0 ** 127, 0x38),
                                      (1.37 * 2.0 ** -95, 0x7E), (2.0 ** -126, 0x7E)])
@each_form
def test_scales_at_the_ends_of_fp32(top, code, Hq, Hkv, D, old, new):
    """Values up to FP32's largest: no sum on the way leaves its range."""
    case = spread(np.random.default_rng(D), old, new, Hq, Hkv, D, 32, lambda e, pages: top)
    v = case[3]
    v[...] = (v & 0x80) | np.minimum(v & 0x7F, code)
    bound_check(case)


def test_one_token_of_the_largest_values():
    """Written by the library: a request's only token comes back as it was, up to the cache's rounding."""
    x = torch.tensor([3.1e38, -3.1e38, 1.0, 2.0 ** 113], device=DEV).repeat(2, 1, 16)           # [2][1][64]
    cache = fp8.kv_cache(2, 1, 16, 64, DEV)
    fp8.fp8_kv_append(x * 2.0 ** -127, x, ints([0, 16]), *cache)
    out = fp8.fp8_kv_attention(torch.ones(2, 1, 64, dtype=torch.bfloat16, device=DEV), *cache, ints([[0], [1]]), ints([0, 1, 2]), ints([1, 1]))
    want = kv.values(host(cache[2]), host(cache[3]), np.array([0]), 1, 16, 0, turned=True)[0]
    assert np.abs(want).max() > 3e38 and np.array_equal(host(out)[0], want) and np.array_equal(host(out)[1], want)


@pytest.mark.parametrize("Hq,Hkv,old,new", [
    (8, 2, [700, 64, 0, 1300, 33, 500], [1, 1, 1, 4, 2, 400]),                # few rows beside a chunk: 128 rows a workgroup, split
    (4, 2, [700, 20, 0, 90, 1100] * 6, [1, 1, 3, 1, 2] * 5 + [1, 1, 3, 1, 150])])      # a chunk beside many: 16 rows
def test_steps_that_mix_single_tokens_and_chunks(Hq, Hkv, old, new):
    """Single tokens, a few drafted ones and a prompt's chunk in one call."""
    case = list(attention_case(np.random.default_rng(Hq), old, new, Hq, Hkv, 64, 32, special=False))
    case[2], case[4] = np.full(case[2].shape, 2.0 ** -8), case[4].astype(np.float64)
    bound_check(case)


def test_a_mixed_step_that_fills_the_chip():
    """Nothing is split there, a long single token neither: what each request gives in a call of its own."""
    q, k, ks, v, vs, table, cu, lens = on_gpu(attention_case(np.random.default_rng(5), [1500, 64, 300, 15], [1, 3, 1, 1160], 64, 64, 64, 32, special=False))
    assert fp8.fp8_kv_attention_workspace(q.shape[0], 4, 64, 64, 64, 32, table.shape[1]) == 0
    lse = torch.empty(q.shape[:2], device=DEV)
    out, _ = fp8.fp8_kv_attention(q, k, ks, v, vs, table, cu, lens, lse=lse)
    at = cu.tolist()
    for b in range(4):
        rows = slice(at[b], at[b + 1])
        alone_lse = torch.empty_like(lse[rows])
        alone, _ = fp8.fp8_kv_attention(q[rows], k, ks, v, vs, table[b: b + 1].clone(), ints([0, at[b + 1] - at[b]]), lens[b: b + 1].clone(), lse=alone_lse)
        # either call is within the bound of the exact result (X < 2^4, n < 2^11: 2^-10 of sum_j p_j |v_j|, at most 448 / 64 here), and rounds once
        lim = 2 * (2.0 ** -10 * 7.0) + 2.0 ** -7 * alone.float().abs()
        assert bool(((out[rows].float() - alone.float()).abs() <= lim).all()), b
        assert bool(((lse[rows] - alone_lse).abs() <= 2.0 ** -10).all()), b
