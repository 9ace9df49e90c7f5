"""The example layer: its training step against automatic differentiation in 64 bits, its serving step
against the layer of the values that its 4-bit operands stand for.

Bounds.  The training step rounds to bf16 (2^-9 of a value) at each of its half a dozen intermediate
tensors: 2^-5 of a gradient's norm is several times their sum.  The router's gradient is a difference,
w_j (dw_j - sum_i w_i dw_i), which may all but cancel (of one token in particular); its roundings are
those of its terms: each slot's dw is off by some 2^-9 of |dy o_j|, o_j the slot's output and the
product taken by element, so there 2^-5 is of w_j (|dy o_j| + sum_i w_i |dy o_i|) times |x|, the root of
the sum of its squares over slots and tokens.  The serving step's two quantisations
of rows are those of the reference here except where an intermediate's rounding to bf16 moves a value
across a code's half way: 2^-5 of the norm again."""

import importlib.util
import os

import pytest
import torch

import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def same_inputs():
    torch.manual_seed(1)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference(x, router, wi, wo, experts, mask=None):
    """The layer in 64 bits with the choice given (-1: none)."""
    took = experts >= 0
    at = experts.clamp(min=0).long()
    logits = (x @ router.T).gather(1, at)
    logits = torch.where(took, logits, torch.full_like(logits, -torch.inf))
    logits = torch.where(took.any(1, keepdim=True), logits, torch.zeros_like(logits))
    w = torch.where(took, torch.softmax(logits, dim=1), torch.zeros_like(logits))
    y = torch.zeros_like(x)
    for e in range(wi.shape[0]):
        t, j = torch.nonzero((experts == e) & took, as_tuple=True)
        if t.numel():
            gate, up = (x[t] @ wi[e].T).chunk(2, dim=1)
            y = y.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ wo[e].T))
    return y


def router_size(x, router, wi, wo, experts, dy):
    """The size of the terms that the router's gradient is the difference of (no slot dropped)."""
    at = experts.long()
    w = torch.softmax((x @ router.T).gather(1, at), dim=1)
    s = torch.zeros_like(w)
    for e in range(wi.shape[0]):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        gate, up = (x[t] @ wi[e].T).chunk(2, dim=1)
        s[t, j] = (dy[t] * ((torch.nn.functional.silu(gate) * up) @ wo[e].T)).norm(dim=1)
    size = w * (s + (w * s).sum(1, keepdim=True))
    return (size.square().sum(1) * x.square().sum(1)).sum().sqrt()


def near(got, want, what, size=None):
    off = (got.double() - want).norm() / (want.norm() if size is None else size)
    assert off < 2.0 ** -5, (what, float(off))


@pytest.mark.parametrize("tokens,experts,d,f,topk", [(1, 8, 128, 64, 2), (300, 16, 256, 128, 4), (1000, 5, 264, 72, 3)])
def test_training_step(example, tokens, experts, d, f, topk):
    layer = example.MoeLayer(experts, d, f, topk)
    x = torch.randn((tokens, d), device="cuda").to(torch.bfloat16)
    mask = torch.rand(tokens, device="cuda") > 0.1
    mask[0] = True
    y, saved = layer.forward(x, mask)
    dy = torch.randn_like(y)
    dx, grads = layer.backward(dy, saved)
    assert (y[~mask] == 0).all() and (dx[~mask] == 0).all()
    leaves = [t.double().requires_grad_() for t in (x, layer.router, layer.wi, layer.wo)]
    want = reference(*leaves, saved[3])
    near(y, want.detach(), "y")
    want.backward(dy.double())
    for got, leaf, what in zip((dx, grads["wi"], grads["wo"]), (leaves[0], *leaves[2:]), ("dx", "wi", "wo")):
        near(got, leaf.grad, what)
    kept = mask.nonzero()[:, 0]
    size = router_size(leaves[0].detach()[kept], *(t.detach() for t in leaves[1:]), saved[3][kept], dy.double()[kept])
    near(grads["router"], leaves[1].grad, "router", size)
    assert G.read_device_errors() == 0


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,experts,d,f,topk", [(1, 8, 256, 128, 2), (64, 64, 512, 256, 4), (700, 6, 288, 160, 3)])
def test_serving_step(example, tokens, experts, d, f, topk, fmt):
    layer = example.MoeLayer(experts, d, f, topk).pack(fmt)
    x = torch.randn((tokens, d), device="cuda").to(torch.bfloat16)
    y = layer.decode(x)
    weights, chosen = G.route(x @ layer.router.T, topk)
    wi, wo = (G.dequantize_fp4(p, torch.float32).double() for p in layer.packed)
    rows = G.dequantize_fp4(G.quantize_fp4(x, fmt), torch.float32).double()
    want = torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
    for e in range(experts):
        t, j = torch.nonzero(chosen == e, as_tuple=True)
        if t.numel():
            h = (rows[t] @ wi[e].T).to(torch.bfloat16)
            act = G.dequantize_fp4(G.quantize_fp4(layer._gate(h), fmt), torch.float32).double()
            want.index_add_(0, t, weights[t, j, None].double() * (act @ wo[e].T))
    near(y, want, fmt)
    assert G.read_device_errors() == 0


def test_the_example_runs(example, capsys):
    example.main()
    assert "decoding step of 64 tokens" in capsys.readouterr().out
