"""The example layer with the losses that balance its experts, and its decoding step of few tokens with weights in
4-bit integers.

Bounds.  The losses' gradient reaches the router and x through two products in bf16: 2^-5 of the norm is several
times their roundings, as for the layer's other gradients.  The decoding step rounds the activations between its
products to bf16 (2^-9 of each, before the second product); 2^-6 of the norm is several times that."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from test_moe_layer_gpu import example, near, same_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,d,f,topk,sequences", [(300, 16, 256, 128, 4, 3), (64, 5, 264, 72, 3, 1)])
def test_training_step_with_balance(example, tokens, experts, d, f, topk, sequences):  # noqa: F811
    layer = example.MoeLayer(experts, d, f, topk)
    x = torch.randn((tokens, d), device="cuda").to(torch.bfloat16)
    mask = torch.rand(tokens, device="cuda") > 0.1
    y, saved = layer.forward(x, mask)
    balance = layer.balance(saved, sequences)
    assert int(balance.counts.sum()) == topk * int(mask.sum()) and int(balance.tokens) == int(mask.sum())
    dlosses = torch.tensor([30.0, 3.0], device="cuda")
    none = torch.zeros_like(y)
    dx, grads = layer.backward(none, saved, balance, dlosses)
    x64, router = x.double().requires_grad_(), layer.router.double().requires_grad_()
    logits = x64 @ router.T
    p = torch.softmax(logits, dim=1)
    share = balance.counts.double() / balance.counts.sum(1, keepdim=True)
    share = share.repeat_interleave(tokens // sequences, dim=0)
    n = mask.sum()
    losses = torch.stack((experts * (share * p).sum(1)[mask].sum() / n, (torch.logsumexp(logits, 1) ** 2)[mask].sum() / n))
    near(balance.losses, losses.detach(), "losses")
    (losses * dlosses.double()).sum().backward()
    near(dx, x64.grad, "dx")
    near(grads["router"], router.grad, "router")
    assert not grads["wi"].any() and not grads["wo"].any()
    # and added to the layer's own
    dy = torch.randn_like(y)
    both, own = layer.backward(dy, saved, balance, dlosses)[1]["router"], layer.backward(dy, saved)[1]["router"]
    near(both.double() - own.double(), router.grad, "sum", router.grad.norm() + own.double().norm())


@pytest.mark.parametrize("fmt", ["int4", "uint4"])
@pytest.mark.parametrize("tokens,experts,d,f,topk", [(1, 8, 256, 128, 2), (7, 64, 512, 256, 4), (40, 6, 320, 192, 3)])
def test_decoding_step_in_integers(example, tokens, experts, d, f, topk, fmt):  # noqa: F811
    layer = example.MoeLayer(experts, d, f, topk).pack(fmt)
    x = torch.randn((tokens, d), device="cuda").to(torch.bfloat16)
    y = layer.decode(x)
    weights, chosen = G.route(x @ layer.router.T, topk)
    wi, wo = (G.dequantize_int4(p, torch.float32).double() for p in layer.packed)
    want = torch.zeros((tokens, d), dtype=torch.float64, device="cuda")
    for e in range(experts):
        t, j = torch.nonzero(chosen == e, as_tuple=True)
        if t.numel():
            gate, up = (x[t].double() @ wi[e].T).chunk(2, dim=1)
            act = gate / (1 + torch.exp(-gate)) * up
            want.index_add_(0, t, weights[t, j, None].double() * (act @ wo[e].T))
    assert (y.double() - want).norm() < 2.0 ** -6 * want.norm()


def test_the_example_prints_both_decoding_steps(example, capsys):  # noqa: F811
    example.main()
    out = capsys.readouterr().out
    assert "decoding step of 64 tokens in mxfp4" in out and "decoding step of 1 tokens in int4" in out and "balance loss" in out
