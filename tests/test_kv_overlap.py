"""Buffers that overlap are refused by the host, before any launch (no GPU needed): waves read what others have written."""
import ctypes

import pytest

from tests.test_kv_abi import EUNSUP, NUL, call

T, D, SIZE = 7, 128, 2                                         # tokens, channels, bytes of BF16
BASE = 0x10000000


def at(i, elements=0):
    """The i-th of buffers far from one another, and so many elements on."""
    return ctypes.c_void_p(BASE + (i << 24) + SIZE * elements)


def rope(**c):
    """4 query heads and 2 key heads, every buffer apart and contiguous."""
    order = "q ldq qo ldqo Hq k ldk ko ldko Hkv bf16 pos freqs T D rot inter scale inv"
    good = dict(q=at(0), ldq=4 * D, qo=at(1), ldqo=4 * D, Hq=4, k=at(2), ldk=2 * D, ko=at(3), ldko=2 * D, Hkv=2, bf16=1, pos=at(4), freqs=at(5),
                T=T, D=D, rot=64, inter=0, scale=1.0, inv=0)
    return call("rope", order, good, **c)


@pytest.mark.parametrize("case", [
    dict(qo=at(0, 4 * D)), dict(qo=at(0, D)), dict(qo=at(0, -D)), dict(qo=at(0, -4 * D)),             # queries a row or a head further
    dict(qo=at(0, (T - 1) * 4 * D + 3 * D)), dict(ko=at(2, 2 * D)), dict(ko=at(2, -8)),
    dict(qo=at(2)), dict(ko=at(0)), dict(qo=at(2, -T * 4 * D + D)), dict(ko=at(0, (T - 1) * 4 * D)),  # on the other's input
    dict(qo=at(0), ko=at(0)), dict(qo=at(1), ko=at(1)), dict(qo=at(1), ko=at(1, T * 4 * D - 8)),      # both outputs on one buffer
    dict(qo=at(0), k=at(0), ko=at(3)), dict(q=at(0), k=at(0), qo=at(0), ko=at(0)),                    # in place on a shared input
    dict(qo=at(4)), dict(ko=at(5)), dict(qo=at(5, -T * 4 * D + 8)), dict(ko=at(4, 8)),                # on positions and frequencies
    # rows of 12 heads of one buffer: queries 0 to 3, keys 4 and 5, outputs that begin a head too early, or run into the next row
    dict(q=at(0), ldq=12 * D, k=at(0, 4 * D), ldk=12 * D, qo=at(0, 5 * D), ldqo=12 * D, ko=at(0, 10 * D), ldko=12 * D),
    dict(q=at(0), ldq=12 * D, k=at(0, 4 * D), ldk=12 * D, qo=at(0, 6 * D), ldqo=12 * D, ko=at(0, 9 * D), ldko=12 * D),
    dict(q=at(0), ldq=12 * D, k=at(0, 4 * D), ldk=12 * D, qo=at(0, 6 * D), ldqo=12 * D, ko=at(0, 11 * D), ldko=12 * D),
    # rows at other distances: the fourth row of one meets the third of the other
    dict(q=at(0), ldq=6 * D, qo=at(0, 4 * D), ldqo=8 * D, Hq=2, ko=at(3))])
def test_rope(case):
    assert rope(**case) == EUNSUP


def test_rope_of_queries_alone():
    none = dict(k=NUL, ko=NUL, Hkv=0)
    assert rope(qo=at(0, 8), **none) == EUNSUP and rope(qo=at(4), **none) == EUNSUP
    assert rope(T=1, qo=at(0, 3 * D), **none) == EUNSUP


def assign(**c):
    names = "have add free nf table lens cu pos slots left".split()
    return call("kv_assign_pages", "have add B free nf F page table width T lens cu pos slots left",
                dict({k: at(i) for i, k in enumerate(names)}, B=4, F=100, page=64, width=8, T=9), **c)


def test_outputs_of_the_page_tables_on_one_another():
    """What one workgroup writes of a buffer another would write as well."""
    for a, b in (("cu", 5), ("pos", 4), ("left", 8), ("slots", 7), ("cu", 4)):
        assert assign(**{a: at(b)}) == EUNSUP, (a, b)
    assert assign(cu=at(7, -8)) == EUNSUP                      # the last of five
    got = call("kv_release_pages", "done lens table B width page free F nf out left",
               dict(done=at(0), lens=at(1), table=at(2), free=at(3), nf=at(4), out=at(3, 192), left=at(5), B=4, width=8, page=64, F=100))
    assert got == EUNSUP


def append(**c):
    return call("fp8_kv_append", "k ldk v ldv bf16 slots T H D page n kc ks vc vs",
                dict(k=at(0), ldk=2 * D, v=at(1), ldv=2 * D, bf16=1, slots=at(2), T=T, H=2, D=D, page=64, n=10, kc=at(3), ks=at(4), vc=at(5), vs=at(6)), **c)


@pytest.mark.parametrize("case", [dict(kc=at(0)), dict(vc=at(1, (T - 1) * 2 * D)), dict(ks=at(0, 2 * D)), dict(vs=at(2)), dict(vc=at(2, -8)),
                                  dict(vc=at(3)), dict(vs=at(4)), dict(vs=at(4, 32)), dict(ks=at(3, 8)), dict(vc=at(3, 10 * 2 * 64 * D // 2 - 8)),
                                  dict(v=at(0, 2 * D), ldk=6 * D, ldv=6 * D, kc=at(0, 4 * D))])
def test_append(case):
    assert append(**case) == EUNSUP


def attend(**c):
    return call("fp8_kv_attention", "q ldq kc ks vc vs n page table width cu lens B T Hq Hkv D scale out lse ws wb",
                dict(q=at(0), ldq=8 * D, kc=at(1), ks=at(2), vc=at(3), vs=at(4), n=10, page=64, table=at(5), width=40, cu=at(6), lens=at(7), B=3, T=T,
                     Hq=8, Hkv=2, D=D, scale=0.1, out=at(8), lse=at(9), ws=at(10), wb=1 << 30), **c)


@pytest.mark.parametrize("case", [dict(out=at(0, 8 * D)), dict(out=at(0, -D)), dict(out=at(0), ldq=9 * D), dict(out=at(1)), dict(out=at(2)), dict(out=at(3)),
                                  dict(out=at(4, 8)), dict(out=at(5)), dict(out=at(6)), dict(out=at(7)), dict(lse=at(0)), dict(lse=at(8)), dict(lse=at(6)),
                                  dict(ws=at(0)), dict(ws=at(8)), dict(ws=at(9)), dict(ws=at(5, 16)), dict(out=at(10, 64)), dict(lse=at(10, 8)), dict(ws=at(3))])
def test_attention(case):
    assert attend(**case) == EUNSUP
