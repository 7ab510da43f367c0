"""Host-side checks of the key/value cache's entry points: bad arguments are
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


def assign(**c):
    return call("kv_assign_pages", "have add B free nf F page table width T lens cu pos slots left",
                dict(have=P, add=P, B=4, free=P, nf=P, F=100, page=64, table=P, width=8, T=9, lens=P, cu=P, pos=P, slots=P, left=P), **c)


def test_assign_refusals():
    for k in ("have", "add", "free", "nf", "table", "lens", "cu", "pos", "slots", "left"):
        assert assign(**{k: NUL}) == ENULL, k
        if k != "nf":
            assert assign(**{k: MIS}) == EALIGN, k
    assert assign(nf=ctypes.c_void_p(0x10002)) == EALIGN
    for bad in (dict(B=-1), dict(width=-1), dict(T=-1), dict(F=-1)):
        assert assign(**bad) == ESHAPE, bad
    for bad in (dict(page=0), dict(page=8), dict(page=48), dict(page=512), dict(B=65537), dict(F=BIG), dict(T=1 << 23),
                dict(B=65536, width=1 << 15), dict(width=1 << 25), dict(page=-16)):
        assert assign(**bad) == EUNSUP, bad


def test_release_refusals():
    def f(**c):
        return call("kv_release_pages", "done lens table B width page free F nf out left",
                    dict(done=P, lens=P, table=P, B=4, width=8, page=64, free=P, F=100, nf=P, out=P, left=P), **c)
    for k in ("done", "lens", "table", "free", "nf", "out", "left"):
        assert f(**{k: NUL}) == ENULL, k
        if k != "nf":
            assert f(**{k: MIS}) == EALIGN, k
    for bad in (dict(B=-1), dict(width=-1), dict(F=-1)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(page=24), dict(B=65537), dict(F=BIG), dict(B=65536, width=1 << 15)):
        assert f(**bad) == EUNSUP, bad


def test_rope_refusals():
    def f(**c):
        return call("rope", "q ldq qo ldqo Hq k ldk ko ldko Hkv bf16 pos freqs T D rot inter scale inv",
                    dict(q=P, ldq=512, qo=P, ldqo=512, Hq=4, k=P, ldk=256, ko=P, ldko=256, Hkv=2, bf16=1, pos=P, freqs=P, T=0, D=128, rot=64,
                         inter=0, scale=1.0, inv=0), **c)
    assert f() == OK and f(T=5, Hq=0, Hkv=0, q=NUL, qo=NUL, k=NUL, ko=NUL) == OK
    assert f(q=NUL, qo=NUL, k=NUL, ko=NUL, pos=NUL, freqs=NUL) == OK                  # T = 0
    for k in ("q", "qo", "k", "ko", "pos", "freqs"):
        assert f(T=2, **{k: NUL}) == ENULL and f(**{k: MIS}) == EALIGN
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(D=0), dict(D=124), dict(rot=0), dict(rot=24), dict(rot=144), dict(rot=-16),
                dict(ldq=511), dict(ldq=516), dict(ldqo=504), dict(ldk=255), dict(ldko=257)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(bf16=2), dict(inter=2), dict(inv=-1), dict(T=BIG), dict(D=512, rot=272, ldq=2048, ldqo=2048, ldk=1024, ldko=1024),
                dict(D=1032, ldq=1 << 20, ldqo=1 << 20, ldk=1 << 20, ldko=1 << 20), dict(Hq=65536, ldq=1 << 24, ldqo=1 << 24),
                dict(T=1 << 30, ldq=1 << 11)):
        assert f(**bad) == EUNSUP, bad


def append(**c):
    return call("fp8_kv_append", "k ldk v ldv bf16 slots T H D page n kc ks vc vs",
                dict(k=P, ldk=256, v=P, ldv=256, bf16=1, slots=P, T=0, H=2, D=128, page=64, n=10, kc=P, ks=P, vc=P, vs=P), **c)


def test_append_refusals():
    assert append() == OK and append(T=4, H=0) == OK and append(T=4, n=0) == OK
    assert append(k=NUL, v=NUL, slots=NUL, kc=NUL, ks=NUL, vc=NUL, vs=NUL) == OK
    for k in ("k", "v", "slots", "kc", "ks", "vc", "vs"):
        assert append(T=1, **{k: NUL}) == ENULL and append(**{k: MIS}) == EALIGN
    for bad in (dict(T=-1), dict(H=-1), dict(n=-1), dict(ldk=255), dict(ldv=260), dict(ldv=128)):
        assert append(**bad) == ESHAPE, bad
    for bad in (dict(bf16=2), dict(D=96), dict(D=0), dict(D=512), dict(page=20), dict(page=512), dict(n=1 << 26), dict(T=BIG),
                dict(H=65536, ldk=1 << 24, ldv=1 << 24), dict(n=1 << 24, H=1 << 10, ldk=1 << 17, ldv=1 << 17)):
        assert append(**bad) == EUNSUP, bad


ORDER = "q ldq kc ks vc vs n page table width cu lens B T Hq Hkv D scale out lse ws wb"
GOOD = dict(q=P, ldq=1024, kc=P, ks=P, vc=P, vs=P, n=10, page=64, table=P, width=4, cu=P, lens=P, B=3, T=0, Hq=8, Hkv=2, D=128, scale=0.1,
            out=P, lse=P, ws=P, wb=1 << 30)


def attend(**c):
    return call("fp8_kv_attention", ORDER, GOOD, **c)


def test_attention_refusals():
    assert attend() == OK and attend(T=4, B=0) == OK and attend(T=4, Hq=0, Hkv=0, n=0) == OK
    for k in ("q", "kc", "ks", "vc", "vs", "table", "cu", "lens", "out"):
        assert attend(T=1, **{k: NUL}) == ENULL, k
    for k in ("q", "kc", "ks", "vc", "vs", "table", "cu", "lens", "out", "lse", "ws"):
        assert attend(**{k: MIS}) == EALIGN, k
    for bad in (dict(T=-1), dict(B=-1), dict(width=-1), dict(Hq=-8), dict(Hkv=-2), dict(Hkv=3), dict(Hkv=0), dict(ldq=1023), dict(ldq=1028),
                dict(n=-1), dict(T=1, n=0)):
        assert attend(**bad) == ESHAPE, bad
    for bad in (dict(D=96), dict(D=320), dict(page=40), dict(page=512), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(T=BIG), dict(B=65537), dict(width=1 << 25), dict(n=1 << 26), dict(T=1 << 30, Hq=1 << 10, Hkv=1, ldq=1 << 17),
                dict(Hq=65536, Hkv=1, ldq=1 << 23)):
        assert attend(**bad) == EUNSUP, bad


def test_attention_workspace():
    f = fp8.fp8_kv_attention_workspace
    assert f(4, 4, 8, 2, 128, 64, 4) == 0                      # 256 tokens: never split
    assert f(0, 4, 8, 2, 128, 64, 1000) == 0 and f(4, 0, 8, 2, 128, 64, 1000) == 0
    need = f(4, 4, 8, 2, 128, 64, 1000)
    assert 0 < need < 1 << 28
    assert attend(T=4, B=4, width=1000, ws=NUL) == ENULL and attend(T=4, B=4, width=1000, wb=need - 1) == ESHAPE
    with pytest.raises(fp8.Fp8fgError):
        f(4, 4, 9, 2, 128, 64, 4)
    assert fp8.load_library().fp8_kv_attention_workspace(4, 4, 8, 2, 128, 64, 4, None) == ENULL


def test_grids_longer_than_a_launch_are_refused():
    """2^32 threads and more along a grid's axis: refused before anything is enqueued."""
    assert append(T=1 << 30, H=1, D=64, ldk=64, ldv=64) == EUNSUP
    assert attend(T=1 << 20, B=1, Hq=64, Hkv=1, D=64, ldq=1 << 12, width=1) == EUNSUP
    assert attend(T=1 << 23, B=1, Hq=65535, Hkv=65535, D=64, ldq=1 << 22, width=1) == EUNSUP        # 65,536 tiles x 65,535 heads


def test_frequencies():
    f, s = fp8.rope_frequencies(8, base=100.0, device="cpu")
    assert s == 1.0 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75]))
    g, s = fp8.rope_frequencies(64, factor=8.0, original=4096, device="cpu")
    f, _ = fp8.rope_frequencies(64, device="cpu")
    turns = f * 4096 / (2 * torch.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 8) and abs(s - 1.2079442) < 1e-6
    assert torch.all((g <= f) & (g >= f / 8.0001))


def test_binding_refuses_what_it_cannot_pass_on():
    x, i = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    cache = fp8.kv_cache(3, 2, 16, 128, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(3, 2, 16, 128), (3, 2), (3, 2, 128, 16), (3, 2)]
    table = torch.zeros(4, 3, dtype=torch.int32)
    for f in (lambda: fp8.kv_assign_pages(i, i, table, i, i[:1], 16, 4), lambda: fp8.kv_release_pages(i, i, table, i, i[:1], 16),
              lambda: fp8.rope(x, None, i, torch.zeros(64)), lambda: fp8.fp8_kv_append(x, x, i, *cache),
              lambda: fp8.fp8_kv_attention(x, *cache, table, i, i)):
        with pytest.raises(ValueError):
            f()


class Elsewhere:
    """A stand-in for a tensor on another device."""
    is_cuda, dtype, shape, device = True, torch.int32, (4,), "cuda:1"

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True


def test_tensors_on_different_devices():
    fp8._need_at(1, Elsewhere(1), torch.int32, (4,), "lens")
    with pytest.raises(ValueError, match="lens must be on device 0"):
        fp8._need_at(0, Elsewhere(1), torch.int32, (4,), "lens")


def test_calls_run_on_the_tensors_device(monkeypatch):
    """The call is made with the tensor's device current, on that device's stream."""
    seen = []

    class Guard:
        def __init__(self, index):
            seen.append(("device", index))

        def __enter__(self):
            seen.append("in")

        def __exit__(self, *a):
            seen.append("out")

    class Library:
        def rope(self, *args):
            seen.append(args)
            return 0

    monkeypatch.setattr(fp8, "load_library", lambda: Library())
    monkeypatch.setattr(fp8, "_current_device", lambda: 0)
    monkeypatch.setattr(fp8, "_stream", lambda t: 70 + t.get_device())
    monkeypatch.setattr(torch.cuda, "device", Guard)
    fp8._run("rope", 2, Elsewhere(2), 5)
    fp8._run("rope", 0, Elsewhere(0), 6)
    assert seen == [("device", 2), "in", (5, 72), "out", (6, 70)]


def test_positions_are_rounded_to_tiles():
    """page * width up to 2^31 - 256, whatever the page."""
    for page in (16, 64, 256):
        most = (2 ** 31 - 256) // page
        for f in (assign, attend):
            assert f(B=1, page=page, width=most + 1) == EUNSUP
        assert attend(B=1, page=page, width=most) == OK


def test_buffers_that_overlap():
    """Outputs on top of inputs are refused: some workgroups would read what others have written."""
    def at(i):
        return ctypes.c_void_p(0x100000 * (i + 1))

    names = ("have", "add", "free", "nf", "table", "lens", "cu", "pos", "slots", "left")
    apart = {k: at(i) for i, k in enumerate(names)}
    for out, inp in (("lens", "have"), ("lens", "add"), ("left", "nf"), ("cu", "add"), ("slots", "free"), ("table", "have"), ("pos", "have")):
        assert assign(**dict(apart, **{out: apart[inp]})) == EUNSUP, (out, inp)
    # the last of four lengths, and of a hundred pages
    assert assign(**dict(apart, cu=ctypes.c_void_p(apart["have"].value - 16))) == EUNSUP
    assert assign(**dict(apart, have=ctypes.c_void_p(apart["free"].value + 384), pos=ctypes.c_void_p(apart["free"].value + 384))) == EUNSUP
    names = ("done", "lens", "table", "free", "nf", "out", "left")
    apart = {k: at(i) for i, k in enumerate(names)}
    for out, inp in (("out", "lens"), ("left", "nf"), ("free", "table"), ("out", "done")):
        got = call("kv_release_pages", "done lens table B width page free F nf out left",
                   dict(apart, B=4, width=8, page=64, F=100, **{out: apart[inp]}))
        assert got == EUNSUP, (out, inp)


def test_rope_in_place_keeps_its_rows():
    order = "q ldq qo ldqo Hq k ldk ko ldko Hkv bf16 pos freqs T D rot inter scale inv"
    good = dict(q=P, ldq=512, qo=P, ldqo=512, Hq=4, k=P, ldk=256, ko=P, ldko=256, Hkv=2, bf16=1, pos=P, freqs=P, T=3, D=128, rot=64, inter=0,
                scale=1.0, inv=0)
    assert call("rope", order, good, ldqo=520) == EUNSUP and call("rope", order, good, ldk=264) == EUNSUP
