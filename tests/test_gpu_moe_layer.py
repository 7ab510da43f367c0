"""The example layer, forward, backward and decode, against plain FP32.

Each product's two operands are rounded to E4M3 (rms relative error near 2.7% each for
normal values, so about 3.8% per product); the output passes two products and
the gate, gradients up to four, with operands rounded twice where they come from a
checkpoint: independent errors add to about 7% and 11%.  The bounds are about twice that."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden,inner,experts,topk,groups,tokens", [(256, 128, 4, 2, 1, 33), (512, 256, 16, 4, 4, 300), (1024, 512, 8, 8, 2, 1000)])
def test_layer(hidden, inner, experts, topk, groups, tokens):
    from examples.moe_layer import MoeLayer, reference, relative
    layer = MoeLayer(hidden, inner, experts, topk, n_groups=groups, topk_groups=groups, scale=2.5, seed=hidden)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    dout = (torch.randn(tokens, hidden, generator=g, device="cuda") * 1e-3).bfloat16()
    out, saved = layer.forward(x)
    grads = layer.backward(dout, saved)
    ref, ref_grads = reference(layer, x, saved[2], dout)
    assert relative(out, ref) < 0.14
    for name, a, b in zip(("x", "router", "gate_up", "down"), grads, ref_grads):
        assert a.shape == b.shape and relative(a, b) < 0.22, name
    again = layer.backward(dout, layer.forward(x)[1])
    assert all(torch.equal(a, b) for a, b in zip(grads[2:], again[2:]))      # the library's own sums repeat bit for bit
    few = x[:40].contiguous()
    step = layer.decode(few, 64)
    assert relative(step, reference(layer, few, layer.route(few)[1])) < 0.14


def test_layer_steps_downhill():
    """A few steps of plain gradient descent with the layer's gradients lower its loss."""
    from examples.moe_layer import MoeLayer
    layer = MoeLayer(256, 128, 8, 2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(512, 256, generator=g, device="cuda").bfloat16()
    target = torch.randn(512, 256, generator=g, device="cuda")
    losses = []
    for _ in range(8):
        out, saved = layer.forward(x)
        diff = out.float() - target
        losses.append(float(diff.square().sum()))
        _, d_router, d_gate_up, d_down = layer.backward(diff.bfloat16(), saved)
        layer.router -= 2e-4 * d_router
        layer.gate_up -= 2e-3 * d_gate_up
        layer.down -= 2e-3 * d_down
        layer.quantize()
    assert losses[-1] < 0.9 * losses[0], losses
