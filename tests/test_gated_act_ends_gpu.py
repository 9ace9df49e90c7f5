"""gated_act() and its gradient with infinities and NaN in either half and in the gradient, for both types: bf16 has an
exponential and a quotient of its own."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


def rows(dtype, f, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    h, d = (torch.randn((6, n), generator=gen, device=DEV).to(dtype) for n in (2 * f, f))
    return h, d


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("f", [32, 37, 1000])
def test_infinities_and_nans_stay_in_their_place(dtype, act, f):
    h, d = rows(dtype, f, f)
    h[h == 0] = 1
    d[d == 0] = 1
    want, back = G.gated_act(h, act), G.gated_act_backward(d, h, act)
    at = {"gate nan": (1, 3, NAN), "up nan": (1, f + 8, NAN), "gate inf": (2, 5, INF), "gate -inf": (2, 9, -INF),
          "up inf": (3, f + 4, INF), "up -inf": (4, 2 * f - 1, -INF)}
    bad = h.clone()
    for r, c, v in at.values():
        bad[r, c] = v
    nan_d = d.clone()
    nan_d[5, 7] = NAN
    out, dh = G.gated_act(bad, act), G.gated_act_backward(nan_d, bad, act)
    touched = torch.zeros_like(out, dtype=torch.bool)
    for r, c, _ in at.values():
        touched[r, c % f] = True
    assert torch.equal(out[~touched], want[~touched])
    touched[5, 7] = True
    both = torch.cat((touched, touched), 1)
    assert torch.equal(dh[~both], back[~both])
    assert out[1, 3].isnan() and out[1, 8].isnan()
    assert out[2, 5] == INF * float(torch.sign(h[2, f + 5]))
    assert out[3, 4] == INF * float(torch.sign(want[3, 4] / h[3, f + 4]))
    assert out[4, f - 1] == -INF * float(torch.sign(want[4, f - 1] / h[4, 2 * f - 1]))
    assert dh[1, 3].isnan() and dh[1, f + 3].isnan() and dh[1, 8].isnan() and dh[1, f + 8] == back[1, f + 8]
    assert dh[2, 5] == d[2, 5] * h[2, f + 5] and dh[2, f + 5] == INF * float(torch.sign(d[2, 5]))  # act' is 1 there
    assert dh[5, 7].isnan() and dh[5, f + 7].isnan()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_gate_of_bf16(dtype, act):
    """All finite gates that bf16 has, up to where gelu's cube leaves fp32: finite, and within a step of the bound."""
    import experts_reference as R

    g = torch.arange(0, 2 ** 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g = g[g.isfinite() & (g.float().abs() < 2.0 ** 40)].to(DEV)
    h = torch.stack((g, torch.ones_like(g))).reshape(1, -1).to(dtype)
    d = torch.ones((1, g.numel()), dtype=dtype, device=DEV)
    out, dh = R.as64(G.gated_act(h, act))[0], R.as64(G.gated_act_backward(d, h, act))[0]
    a, slope, x, slopes = R.act(R.as64(g), act)
    with np.errstate(over="ignore"):
        rel = (16 + 8 * np.abs(x)) * R.U32
    half, tiny = R.half_step(dtype) * (1 + 2.0 ** -8), 2.0 ** -126
    n = g.numel()
    assert (np.abs(out - a) <= rel * np.abs(a) + half * np.abs(a) + tiny).all()
    assert (np.abs(dh[:n] - slope) <= rel * slopes + half * np.abs(slope) + tiny).all()
    assert (np.abs(dh[n:] - a) <= rel * np.abs(a) + half * np.abs(a) + tiny).all()
