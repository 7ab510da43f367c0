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
