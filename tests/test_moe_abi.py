"""Host-side checks of the mixture-of-experts entry points: bad arguments are
refused before any launch, empty problems are no-ops (no GPU needed)."""
import ctypes

import pytest
import torch

import fp8_fine_grained_amd as fp8

OK, ENULL, ESHAPE, EALIGN, EUNSUP = 0, -1, -2, -3, -4
P = ctypes.c_void_p(0x10000)          # fake, 16-byte aligned "device" pointer (never dereferenced)
MIS = ctypes.c_void_p(0x10004)
NUL = ctypes.c_void_p(0)
BIG = 1 << 31


def call(name, order, good, **change):
    args = dict(good, **change)
    return getattr(fp8.load_library(), name)(*(args[k] for k in order.split()), NUL)


def route(**c):
    return call("moe_route", "x bf16 ld bias T E topk ng tg top score renorm scale idx w",
                dict(x=P, bf16=0, ld=64, bias=P, T=0, E=64, topk=4, ng=4, tg=2, top=2, score=1, renorm=1, scale=1.0, idx=P, w=P), **c)


def test_route_refusals():
    assert route() == OK                                     # T = 0: no launch
    assert route(bias=NUL, x=NUL, idx=NUL, w=NUL) == OK
    for k in ("x", "idx", "w"):
        assert route(T=1, **{k: NUL}) == ENULL
    for bad in (dict(T=-1), dict(topk=0), dict(E=12, topk=7), dict(ld=63), dict(E=0), dict(ng=3), dict(ng=0), dict(tg=0),
                dict(tg=5), dict(E=8, ng=8, tg=2, topk=3, ld=8)):
        assert route(**bad) == ESHAPE, bad
    for k in ("x", "bias", "idx", "w"):
        assert route(**{k: MIS}) == EALIGN
    for bad in (dict(bf16=2), dict(top=0), dict(top=3), dict(score=2), dict(renorm=-1), dict(T=BIG), dict(topk=17, tg=4),
                dict(E=1025, ld=1025, ng=1, tg=1), dict(E=320, ld=320, ng=32, tg=2), dict(E=1020, ld=1020, ng=5, tg=2)):
        assert route(**bad) == EUNSUP, bad


def test_route_backward_refusals():
    def f(**c):
        return call("moe_route_backward", "x bf16 ld idx dw T E topk score renorm scale dx",
                    dict(x=P, bf16=0, ld=64, idx=P, dw=P, T=0, E=64, topk=4, score=0, renorm=1, scale=1.0, dx=P), **c)
    assert f() == OK and f(x=NUL, idx=NUL, dw=NUL, dx=NUL) == OK
    for k in ("x", "idx", "dw", "dx"):
        assert f(T=1, **{k: NUL}) == ENULL and f(**{k: MIS}) == EALIGN
    for bad in (dict(T=-1), dict(topk=0), dict(topk=65), dict(ld=5)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(score=5), dict(renorm=2), dict(bf16=3), dict(E=2000, ld=2000), dict(topk=20)):
        assert f(**bad) == EUNSUP, bad


def test_dispatch_refusals():
    def c(**k):
        return call("fp8_moe_dispatch_contiguous", "x bf16 T H idx topk first G R q s row off cnt",
                    dict(x=P, bf16=1, T=8, H=64, idx=P, topk=2, first=0, G=0, R=2048, q=P, s=P, row=P, off=P, cnt=P), **k)

    def m(**k):
        return call("fp8_moe_dispatch_masked", "x bf16 T H idx topk first G M q s row mm",
                    dict(x=P, bf16=1, T=8, H=64, idx=P, topk=2, first=0, G=0, M=16, q=P, s=P, row=P, mm=P), **k)
    for f in (c, m):
        assert f() == OK                                     # G = 0: no launch
        for k in ("x", "idx", "q", "s", "row"):
            assert f(G=4, **{k: NUL}) == ENULL
            assert f(G=4, **{k: MIS}) == EALIGN
        for bad in (dict(H=24), dict(T=-1), dict(topk=0), dict(G=-1), dict(H=-16)):
            assert f(**bad) == ESHAPE, bad
        for bad in (dict(topk=17), dict(G=257, R=1 << 20), dict(first=-1), dict(first=BIG), dict(bf16=2), dict(T=BIG, R=BIG - 128)):
            bad = {k: v for k, v in bad.items() if k != "R" or f is c}
            assert f(**bad) == EUNSUP, bad
    assert c(G=4, off=NUL) == ENULL and c(G=4, cnt=NUL) == ENULL and m(G=4, mm=NUL) == ENULL
    assert c(R=2000) == ESHAPE
    assert c(G=4, R=384) == ESHAPE                           # 16 entries of 4 experts may need 4 tiles
    assert fp8.moe_rows_bound(8, 2, 4) == 512 and fp8.moe_rows_bound(1, 1, 4) == 128 and fp8.moe_rows_bound(0, 8, 4) == 0
    assert m(M=0) == ESHAPE and m(G=256, M=1 << 23) == EUNSUP


def test_combine_refusals():
    def f(**k):
        return call("moe_combine", "y bf16 R H row w T topk out dt",
                    dict(y=P, bf16=1, R=128, H=64, row=P, w=P, T=0, topk=2, out=P, dt=0), **k)
    assert f() == OK and f(H=0, T=4) == OK
    for k in ("y", "row", "out"):
        assert f(T=4, **{k: NUL}) == ENULL
    for k in ("y", "row", "w", "out"):
        assert f(**{k: MIS}) == EALIGN
    for bad in (dict(H=20), dict(T=-1), dict(R=-1), dict(topk=0)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(dt=2), dict(bf16=5), dict(topk=17), dict(R=BIG)):
        assert f(**bad) == EUNSUP, bad

    def b(**k):
        return call("fp8_moe_combine_backward", "d db T H y yb R row w topk off cnt G q s dw",
                    dict(d=P, db=1, T=0, H=64, y=P, yb=1, R=128, row=P, w=P, topk=2, off=P, cnt=P, G=0, q=P, s=P, dw=P), **k)
    assert b() == OK
    for k in ("d", "y", "row", "w", "off", "cnt", "q", "s", "dw"):
        assert b(T=4, G=2, **{k: NUL}) == ENULL, k
        assert b(**{k: MIS}) == EALIGN, k
    for bad in (dict(H=24), dict(T=-1), dict(R=-1), dict(topk=0), dict(G=-1)):
        assert b(**bad) == ESHAPE, bad
    for bad in (dict(db=2), dict(yb=2), dict(topk=17), dict(G=257)):
        assert b(**bad) == EUNSUP, bad


def test_swiglu_refusals():
    def f(**k):
        return call("fp8_swiglu", "gu bf16 G M I rows q s qc sc",
                    dict(gu=P, bf16=1, G=1, M=0, I=128, rows=P, q=P, s=P, qc=P, sc=P), **k)
    assert f() == OK and f(G=0, M=4) == OK and f(I=0, M=4) == OK
    for k in ("gu", "q", "s", "qc", "sc"):                   # a checkpoint comes with its scales
        assert f(M=4, **{k: NUL}) == ENULL and f(**{k: MIS}) == EALIGN
    assert f(rows=ctypes.c_void_p(0x10002)) == EALIGN and f(rows=MIS) == OK
    for bad in (dict(I=64), dict(I=200), dict(M=-1), dict(G=-1)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(bf16=2), dict(G=65536), dict(M=BIG), dict(I=(1 << 23) + 128)):
        assert f(**bad) == EUNSUP, bad

    def b(**k):
        return call("fp8_swiglu_backward", "qc sc dh bf16 M I rows q s qt st qh sh",
                    dict(qc=P, sc=P, dh=P, bf16=1, M=0, I=128, rows=P, q=P, s=P, qt=P, st=P, qh=P, sh=P), **k)
    assert b() == OK
    for k in ("qc", "sc", "dh", "q", "s", "qt", "st", "qh", "sh"):
        assert b(M=16, **{k: NUL}) == ENULL and b(**{k: MIS}) == EALIGN
    for bad in (dict(I=64), dict(M=8), dict(M=-16)):
        assert b(**bad) == ESHAPE, bad
    for bad in (dict(bf16=2), dict(M=128 * 65536), dict(I=(1 << 23) + 128)):
        assert b(**bad) == EUNSUP, bad


def test_wgrad_refusals():
    def f(**k):
        return call("fp8_grouped_gemm_wgrad", "a sa b sb off G M N R c acc",
                    dict(a=P, sa=P, b=P, sb=P, off=P, G=0, M=64, N=256, R=256, c=P, acc=0), **k)
    assert f() == OK and f(G=2, M=0) == OK and f(G=2, N=0) == OK
    for k in ("a", "sa", "b", "sb", "off", "c"):
        assert f(G=2, **{k: NUL}) == ENULL and f(**{k: MIS}) == EALIGN
    for bad in (dict(R=100), dict(N=100), dict(M=-1), dict(G=-1), dict(R=-128)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(acc=2), dict(M=BIG), dict(G=1 << 30, M=4096, N=4096)):
        assert f(**bad) == EUNSUP, bad


def test_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(4, 128)
    for f in (lambda: fp8.moe_route(x, 2), lambda: fp8.fp8_swiglu(x), lambda: fp8.moe_combine(x, torch.zeros(4, 2, dtype=torch.int32)),
              lambda: fp8.fp8_moe_dispatch_masked(x, torch.zeros(4, 2, dtype=torch.int32), 4, 8),
              lambda: fp8.fp8_grouped_gemm_wgrad(x, x, x, x, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            f()
