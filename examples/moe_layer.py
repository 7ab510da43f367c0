"""A mixture-of-experts feed-forward layer on one GPU, made of the library's calls.

Training keeps 8-bit checkpoints only: the experts' input rows (the FP8 rows that
the dispatch wrote) and the gate's input (written beside the gate's output).  The
backward pass forms every other operand from them.

    python examples/moe_layer.py        # forward, backward and a decode step against plain FP32
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_amd as fp8  # noqa: E402


def quantize_experts(w):
    """FP32 weights [G][N][K] -> codes and scales for the product with w and for the one with its transpose."""
    plain = [fp8.fp8_quant_weight_128x128(e) for e in w]
    turned = [fp8.fp8_quant_weight_128x128(e, transpose_out=True) for e in w]
    return [torch.stack(t) for p in (plain, turned) for t in zip(*p)]


class MoeLayer:
    """`experts` gated feed-forward networks hidden -> inner -> hidden, topk of them per token."""

    def __init__(self, hidden, inner, experts, topk, n_groups=1, topk_groups=1, scale=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma):
            return torch.randn(*shape, generator=g, device="cuda") * sigma

        self.experts, self.topk, self.scale = experts, topk, scale
        self.groups = dict(n_groups=n_groups, topk_groups=topk_groups, group_top=2)
        self.router = normal(experts, hidden, sigma=hidden ** -0.5)
        self.balance = normal(experts, sigma=0.01)
        self.gate_up = normal(experts, 2 * inner, hidden, sigma=hidden ** -0.5)
        self.down = normal(experts, hidden, inner, sigma=inner ** -0.5)
        self.quantize()

    def quantize(self):
        """The FP8 weights of both passes, after each change of the FP32 ones."""
        self.gu, self.gu_s, self.gu_t, self.gu_ts = quantize_experts(self.gate_up)
        self.dn, self.dn_s, self.dn_t, self.dn_ts = quantize_experts(self.down)

    def route(self, x):
        logits = x.float() @ self.router.t()
        return logits, *fp8.moe_route(logits, self.topk, self.balance, score=fp8.SCORE_SIGMOID, scale=self.scale, **self.groups)

    def forward(self, x):
        """x bf16 [T][hidden] -> (out bf16 [T][hidden], what the backward pass needs)."""
        logits, idx, w = self.route(x)
        q, s, row_of, offsets, counts = fp8.fp8_moe_dispatch_contiguous(x, idx, self.experts)
        used = offsets[self.experts:]
        gu = fp8.fp8_grouped_gemm_contiguous(q, s, self.gu, self.gu_s, offsets)
        h, hs, qc, sc = fp8.fp8_swiglu(gu, used, checkpoint=True)
        y = fp8.fp8_grouped_gemm_contiguous(h, hs, self.dn, self.dn_s, offsets)
        out = fp8.moe_combine(y, row_of, w)
        return out, (x, logits, idx, w, q, s, row_of, offsets, counts, qc, sc, y)

    def backward(self, dout, saved):
        """dout bf16 [T][hidden] -> gradients of x, router, gate_up and down."""
        x, logits, idx, w, q, s, row_of, offsets, counts, qc, sc, y = saved
        dy, dys, dw = fp8.fp8_moe_combine_backward(dout, y, row_of, w, offsets, counts)
        dh = fp8.fp8_grouped_gemm_contiguous(dy, dys, self.dn_t, self.dn_ts, offsets)
        dg, dgs, dgt, dgts, ht, hts = fp8.fp8_swiglu_backward(qc, sc, dh, offsets[self.experts:])
        d_down = fp8.fp8_grouped_gemm_wgrad(*fp8.fp8_requant_act_tokenwise(dy, dys), ht, hts, offsets)
        d_gate_up = fp8.fp8_grouped_gemm_wgrad(dgt, dgts, *fp8.fp8_requant_act_tokenwise(q, s), offsets)
        rows = fp8.fp8_grouped_gemm_contiguous(dg, dgs, self.gu_t, self.gu_ts, offsets)
        dx = fp8.moe_combine(rows, row_of, out_dtype=torch.float32)
        dlogits = fp8.moe_route_backward(logits, idx, dw, fp8.SCORE_SIGMOID, True, self.scale)
        return dx + dlogits @ self.router, dlogits.t() @ x.float(), d_gate_up, d_down

    def decode(self, x, m_max=128):
        """One serving step of a few tokens x bf16 [T][hidden], T <= m_max, on the masked layout."""
        _, idx, w = self.route(x)
        q, s, row_of, masked_m = fp8.fp8_moe_dispatch_masked(x, idx, self.experts, m_max)
        gu = fp8.fp8_grouped_gemm_masked(q, s, self.gu, self.gu_s, masked_m)
        h, hs = fp8.fp8_swiglu(gu, masked_m)
        y = fp8.fp8_grouped_gemm_masked(h, hs, self.dn, self.dn_s, masked_m)
        return fp8.moe_combine(y, row_of, w)


def reference(layer, x, idx, dout=None):
    """The same layer in plain FP32 for the choice idx: the output, and the gradients through autograd."""
    x = x.float().requires_grad_()
    router, gate_up, down = (p.clone().requires_grad_() for p in (layer.router, layer.gate_up, layer.down))
    s = torch.sigmoid(x @ router.t()).gather(1, idx.long())
    w = layer.scale * s / s.sum(1, keepdim=True)
    inner = down.shape[2]
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        gu = x[t] @ gate_up[e].t()
        h = torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
        out = out.index_add(0, t, w[t, j, None] * (h @ down[e].t()))
    if dout is None:
        return out.detach()
    return out.detach(), torch.autograd.grad(out, (x, router, gate_up, down), dout.float())


def relative(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def main():
    layer = MoeLayer(hidden=1024, inner=512, experts=16, topk=4, n_groups=4, topk_groups=2, scale=2.5)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1000, 1024, generator=g, device="cuda").bfloat16()
    dout = (torch.randn(1000, 1024, generator=g, device="cuda") * 1e-3).bfloat16()
    out, saved = layer.forward(x)
    grads = layer.backward(dout, saved)
    ref, ref_grads = reference(layer, x, saved[2], dout)
    print("relative difference from FP32: output %.3f" % relative(out, ref), end="")
    for name, a, b in zip(("x", "router", "gate_up", "down"), grads, ref_grads):
        print(", d %s %.3f" % (name, relative(a, b)), end="")
    few = x[:64].contiguous()
    print("; decode %.3f" % relative(layer.decode(few), reference(layer, few, layer.route(few)[1])))


if __name__ == "__main__":
    main()
