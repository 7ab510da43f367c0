"""How many kernels a dispatch launches, counted in a captured graph: one where few workgroups
count the entries, two (the layout once, then the rows) where many would; the same rows either way."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_fine_grained_amd as fp8
from oracle import moe, quant

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def launches(call):
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t(0)
    get = fp8.load_library().hipGraphGetNodes              # the library's own HIP runtime
    get.argtypes, get.restype = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int
    assert get(graph.raw_cuda_graph(), None, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("T,H,topk,E,contiguous,masked", [(1, 7168, 8, 32, 1, 1), (128, 7168, 8, 32, 1, 1), (400, 7168, 4, 16, 1, 1),
                                                          (512, 7168, 2, 8, 2, 1), (1024, 7168, 2, 8, 2, 2), (2048, 7168, 1, 8, 2, 2),
                                                          (2000, 1024, 1, 8, 2, 1), (1500, 2048, 1, 8, 1, 1), (257, 7168, 8, 32, 2, 2)])
def test_launches(T, H, topk, E, contiguous, masked):
    rng = np.random.default_rng(T)
    x = torch.randn(T, H, device=DEV)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :topk].astype(np.int32)
    idx = torch.from_numpy(ids).to(DEV)
    M = max(8, T * topk // E)
    assert launches(lambda: fp8.fp8_moe_dispatch_contiguous(x, idx, E)) == contiguous
    assert launches(lambda: fp8.fp8_moe_dispatch_masked(x, idx, E, M)) == masked
    eq, es = quant.quant_act_1x128(x.cpu().numpy())
    q, s, row, off, cnt = (t.cpu().numpy() for t in fp8.fp8_moe_dispatch_contiguous(x, idx, E))
    want = moe.rows_contiguous(ids, 0, E)
    assert np.array_equal(row, want[0]) and np.array_equal(off, want[1]) and np.array_equal(cnt, want[2])
    for j in range(topk):
        assert np.array_equal(q[row[:, j]], eq) and np.array_equal(s[:, row[:, j]], es)
    q, s, row, mm = (t.cpu().numpy() for t in fp8.fp8_moe_dispatch_masked(x, idx, E, M))
    want = moe.rows_masked(ids, 0, E, M)
    assert np.array_equal(row, want[0]) and np.array_equal(mm, want[1])
    t, j = np.nonzero(row >= 0)
    r = row[t, j]
    assert np.array_equal(q.reshape(E * M, H)[r], eq[t]) and np.array_equal(s[r // M, :, r % M], es[:, t].T)
