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
