"""gated_act() and its gradient against the 64-bit statement.

Bounds, in units u = 2^-24.  The argument x of g / (1 + exp(-x)) has a few roundings, 8 |x| u, which move the
exponential by as much relatively; the exponential, the sum and the quotient add less than 16 u.  The slope is a
sum of two terms with these errors each.  The rounding to the output's type is half a step, its least number is
that of fp32's or bf16's subnormals."""

import numpy as np
import pytest
import torch

import experts_reference as R
import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TINY = 2.0 ** -126


def check(h, dout, act):
    out = G.gated_act(h, act)
    dh = G.gated_act_backward(dout, h, act)
    torch.cuda.synchronize()
    assert out.dtype == h.dtype and dh.dtype == h.dtype and dh.is_contiguous()
    f = h.shape[1] // 2
    g, u, d = R.as64(h[:, :f]), R.as64(h[:, f:]), R.as64(dout)
    a, slope, x, slopes = R.act(g, act)
    rel, half = (16 + 8 * np.abs(x)) * R.U32, R.half_step(h.dtype) * (1 + 2.0 ** -8)

    def near(got, want, size):
        assert (np.abs(R.as64(got) - want) <= rel * size + half * np.abs(want) + TINY).all()

    near(out, a * u, np.abs(a * u))
    near(dh[:, :f], d * u * slope, np.abs(d * u) * slopes)
    near(dh[:, f:], d * a, np.abs(d * a))
    return out, dh


SHAPES = [(1, 1), (1, 8), (3, 5), (17, 64), (64, 1024), (130, 1027), (33, 2052), (9, 4098), (5, 700), (257, 6), (2, 40000)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_value_and_gradient(shape, dtype, act):
    rows, f = shape
    gen = torch.Generator(device=DEV).manual_seed(rows + f)
    h = 3 * torch.randn((rows, 2 * f), generator=gen, device=DEV)
    h[rows // 2:, : f // 2 + 1] *= 10
    check(h.to(dtype), torch.randn((rows, f), generator=gen, device=DEV).to(dtype), act)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pitch,offset", [(128, 0), (136, 0), (132, 4), (130, 2), (129, 1)])
def test_rows_with_a_pitch(pitch, offset, dtype):
    gen = torch.Generator(device=DEV).manual_seed(pitch)
    wide = torch.randn((37 * pitch + 8), generator=gen, device=DEV).to(dtype)
    h = wide[offset:].as_strided((37, 128), (pitch, 1))
    out, dh = check(h, torch.randn((37, 64), generator=gen, device=DEV).to(dtype), "silu")
    dense = h.contiguous()
    assert torch.equal(out, G.gated_act(dense)) and out.shape == (37, 64)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_far_ends(act, dtype):
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 60.0, -60.0, 88.0, -88.0, 200.0, -200.0, 1e4, -1e4, 1e9, -1e9,
                      16.6, -16.6, 4.4, -4.4], device=DEV)
    h = torch.stack((g, torch.full_like(g, 1.5)), 0).reshape(1, -1).to(dtype)
    check(h, torch.full((1, len(g)), 0.75, device=DEV).to(dtype), act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_infinities_and_nans_stay_in_their_place(act):
    h = torch.ones((4, 64), device=DEV)
    h[1, 3], h[1, 40], h[2, 5] = float("nan"), float("nan"), float("inf")
    out = G.gated_act(h, act)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 3] = bad[1, 8] = True
    assert torch.equal(out.isnan(), bad) and out[2, 5] == float("inf") and out[0].isfinite().all()


def test_no_rows_and_rows_of_zeros():
    assert G.gated_act(torch.empty((0, 16), device=DEV)).shape == (0, 8)
    assert G.gated_act_backward(torch.empty((0, 8), device=DEV), torch.empty((0, 16), device=DEV)).shape == (0, 16)
    h = torch.zeros((5, 16), device=DEV)
    assert not G.gated_act(h).any() and not G.gated_act_backward(torch.ones((5, 8), device=DEV), h).any()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """Central differences in 64 bits: h^2 / 6 times a third derivative (below 3 here) and 2^-52 / h."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    h, d = torch.randn((6, 10), generator=gen, device=DEV), torch.randn((6, 5), generator=gen, device=DEV)
    got, h64, d64, step = R.as64(G.gated_act_backward(d, h, act)), R.as64(h), R.as64(d), 1e-4

    def value(v):
        return (R.act(v[:, :5], act)[0] * v[:, 5:] * d64).sum()

    for at in np.ndindex(6, 10):
        hi, lo = h64.copy(), h64.copy()
        hi[at] += step
        lo[at] -= step
        assert abs(got[at] - (value(hi) - value(lo)) / (2 * step)) < 3e-6
