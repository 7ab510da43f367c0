"""A decode step of the mixture-of-experts operators, captured and replayed: every output, rows in use compared."""
import pytest
import torch

import fp8_fine_grained_amd as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_every_output_of_a_replayed_step():
    T, E, H, I, M = 24, 16, 256, 128, 12                   # buffers of 12 rows: some entries find no row
    g = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.randn(T, E, generator=g, device=DEV)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    gu = torch.randn(E, M, 2 * I, generator=g, device=DEV).bfloat16()
    y = torch.randn(E, M, H, generator=g, device=DEV).bfloat16()

    def step():
        idx, w = fp8.moe_route(logits, 4, n_groups=4, topk_groups=3, group_top=2)
        q, s, row, mm = fp8.fp8_moe_dispatch_masked(x, idx, E, M)
        h, hs = fp8.fp8_swiglu(gu, mm)
        return idx, w, row, mm, fp8.moe_combine(y, row, w), q, s, h, hs

    def rows_in_use(out):
        mm = out[3]
        live = torch.arange(M, device=DEV) < mm[:, None]
        q, s, h, hs = out[5:]
        return list(out[:5]) + [q[live], s.transpose(1, 2)[live], h[live], hs.transpose(1, 2)[live]]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    seen = set()
    for k in range(5):
        logits.copy_(torch.randn(T, E, generator=g, device=DEV))
        x.copy_(torch.randn(T, H, generator=g, device=DEV))
        gu.copy_(torch.randn(E, M, 2 * I, generator=g, device=DEV))
        y.copy_(torch.randn(E, M, H, generator=g, device=DEV))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = step()
        for n, (a, b) in enumerate(zip(rows_in_use(got), rows_in_use(want))):
            assert torch.equal(a, b), (k, n)
        seen.add(tuple(got[3].tolist()))
    assert len(seen) > 1                                   # the replays had different rows in use
