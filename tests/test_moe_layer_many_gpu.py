"""The example layer's serving step in 4-bit integers on both sides of the number of tokens where it changes from
matvec_int4() to the sorted rows.

Bounds.  The sorted rows' weights are rounded to bf16 (2^-9 of each), the activations between the products and the
experts' outputs too: 2^-6 of the norm is several times that, as for the step of few tokens."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from test_moe_layer_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int4", "uint4"])
@pytest.mark.parametrize("experts,d,f,topk", [(8, 256, 128, 2), (6, 320, 192, 3)])
def test_few_tokens_and_many_agree(example, experts, d, f, topk, fmt):  # noqa: F811
    layer = example.MoeLayer(experts, d, f, topk).pack(fmt)
    few = layer.FEW
    x = torch.randn((few + 1, d), device="cuda").to(torch.bfloat16)
    many, fewer = layer.decode(x), layer.decode(x[:few])
    weights, chosen = G.route(x @ layer.router.T, topk)
    wi, wo = (G.dequantize_int4(p, torch.float32).double() for p in layer.packed)
    want = torch.zeros((few + 1, d), dtype=torch.float64, device="cuda")
    for e in range(experts):
        t, j = torch.nonzero(chosen == e, as_tuple=True)
        if t.numel():
            gate, up = (x[t].double() @ wi[e].T).chunk(2, dim=1)
            want.index_add_(0, t, weights[t, j, None].double() * (gate / (1 + torch.exp(-gate)) * up @ wo[e].T))
    assert (many.double() - want).norm() < 2.0 ** -6 * want.norm()
    assert (fewer.double() - want[:few]).norm() < 2.0 ** -6 * want[:few].norm()


def test_many_tokens_do_not_call_the_products_of_few(example, monkeypatch):  # noqa: F811
    layer = example.MoeLayer(8, 256, 128, 2).pack("int4")
    called = []
    monkeypatch.setattr(example.G, "matvec_int4", lambda *a, **k: called.append(1))
    layer.decode(torch.randn((layer.FEW + 1, 256), device="cuda").to(torch.bfloat16))
    assert not called
