"""Host-side limits of the mixture-of-experts entry points (no GPU needed)."""
import ctypes

import fp8_fine_grained_amd as fp8

OK, ESHAPE, EUNSUP = 0, -2, -4
P = ctypes.c_void_p(0x10000)          # fake, 16-byte aligned "device" pointer (never dereferenced)
NUL = ctypes.c_void_p(0)


def test_no_local_expert_needs_no_rows():
    assert fp8.moe_rows_bound(100, 8, 0) == 0 and fp8.moe_rows_bound(100, 8, 1) == 896
    lib = fp8.load_library()
    for rows in (0, 128):
        assert lib.fp8_moe_dispatch_contiguous(P, 0, 100, 64, P, 8, 0, 0, rows, P, P, P, P, P, NUL) == OK
    assert lib.fp8_moe_dispatch_contiguous(P, 0, 100, 64, P, 8, 0, 1, 0, P, P, P, P, P, NUL) == ESHAPE


def test_grids_longer_than_a_launch_are_refused():
    """2^32 threads and more along a grid's axis: an unsupported size, refused before anything is enqueued."""
    lib = fp8.load_library()
    T = 1 << 27
    assert lib.moe_route(P, 0, 1024, NUL, T, 1024, 8, 8, 4, 2, 1, 1, 1.0, P, P, NUL) == EUNSUP
    assert lib.moe_route(P, 1, 64, NUL, 1 << 28, 64, 4, 1, 1, 1, 0, 1, 1.0, P, P, NUL) == EUNSUP
    assert lib.moe_route_backward(P, 0, 512, P, P, T, 512, 4, 0, 1, 1.0, P, NUL) == EUNSUP
    assert lib.fp8_moe_dispatch_contiguous(P, 1, T, 512, P, 1, 0, 1, T + 128, P, P, P, P, P, NUL) == EUNSUP
    assert lib.fp8_moe_dispatch_masked(P, 1, T, 512, P, 1, 0, 1, 64, P, P, P, P, NUL) == EUNSUP
    assert lib.moe_combine(P, 1, 1, 512, P, P, T, 1, P, 0, NUL) == EUNSUP
    assert lib.fp8_moe_combine_backward(P, 1, T, 512, P, 1, 1, P, P, 1, P, P, 1, P, P, P, NUL) == EUNSUP
    assert lib.fp8_grouped_gemm_wgrad(P, P, P, P, P, 1 << 24, 1, 16, 128, P, 0, NUL) == EUNSUP
