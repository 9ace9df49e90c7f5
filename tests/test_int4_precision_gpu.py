"""Products with 4-bit integer weights where a sum's terms are of very different sizes, against the 64-bit statement.

Bounds.  The terms of a sum are scale (code - zero) x, their products exact: experts_reference.matvec_adds() units of
2^-23 of sum |w x|, whatever x meets a weight of 0.  A row is brought to 2^90 .. 2^92 and codes to units of 2^-110,
so fp32's least number, 2^-149, is at most 2^-129 of the row's largest |x|: each of these roundings, before and
after the scale, adds that much absolutely."""

import numpy as np
import pytest
import torch

import experts_reference as R
import moe_grouped_matrix_gb300 as G
from test_int4_gpu import BOTH, DEV, choose, make, normal

pytestmark = pytest.mark.gpu
GROUPS = [32, 64, 128]


def near(out, x, w, experts, weights=None, act=None):
    want, size = R.matvec(R.as64(x), R.values(w), experts.cpu().numpy(), None if weights is None else R.as64(weights), act)
    adds = R.matvec_adds(x.shape[-1], w.group)
    top = np.abs(R.as64(x)).max() * (1 if weights is None else np.abs(R.as64(weights)).sum(1).max())
    tol = adds * 2.0 ** -23 * size + R.half_step(out.dtype) * np.abs(want) + 2.0 ** -126
    if act is None:
        tol = tol + adds * (1 + float(w.scale.float().abs().max())) * 2.0 ** -129 * top
    assert (np.abs(R.as64(out) - want) <= tol).all()


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("power", [10, 16, 24, 60])
def test_a_channel_far_above_the_others_that_meets_weights_of_zero(power, group, zero_points):
    """Activations have such channels.  Tokens for each of the ways x comes from: few, many, summed."""
    w = normal((3, 64, 2048), 1, 0.05)
    w[:, :, 77] = 0
    w[1, :, 1290] = 0
    w = G.quantize_int4(w, group, zero_points)
    for tokens in (2, 60):
        x = normal((tokens, 2048), 2, dtype=torch.bfloat16)
        x[:, 77] *= 2.0 ** power
        x[::2, 1290] *= -(2.0 ** power)
        experts, weights = choose(tokens, 3, 2, 3), normal((tokens, 2), 4)
        near(G.matvec_int4(x, w, experts, out_dtype=torch.float32), x, w, experts)
        near(G.matvec_int4(x, w, experts, weights, out_dtype=torch.float32), x, w, experts, weights)
        near(G.matvec_int4(x, w, experts, act="silu", out_dtype=torch.float32), x, w, experts, act="silu")


@pytest.mark.parametrize("zero_points", BOTH)
def test_a_channel_far_above_the_others_in_large_matrices(zero_points):
    """The way that copies an item's x."""
    w = normal((8, 4096, 2176), 1, 0.05)
    w[:, :, 900] = 0
    w = G.quantize_int4(w, 128, zero_points)
    x = normal((40, 2176), 2, dtype=torch.bfloat16)
    x[:, 900] *= 2.0 ** 20
    experts = choose(40, 8, 2, 3)
    near(G.matvec_int4(x, w, experts, out_dtype=torch.float32), x, w, experts)


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("power", [-40, -100, -108, -115, -125, -140])
def test_values_far_below_their_rows_largest(power, group, zero_points):
    """The largest values meet groups whose scale is 0, so that nothing else hides what becomes of the others."""
    w = normal((2, 48, 512), 1, 0.4)
    w[:, :, :256] = 0
    w = G.quantize_int4(w, group, zero_points)
    x = normal((5, 512), 2)
    x[:, :256] *= 2.0 ** 60
    x[:, 256:] *= 2.0 ** (60 + power)
    x = x.to(torch.bfloat16)
    experts = choose(5, 2, 2, 1, 0.0)
    out = G.matvec_int4(x, w, experts, out_dtype=torch.float32)
    near(out, x, w, experts)
    if power >= -100:  # the absolute part of the bound is far below these
        want, size = R.matvec(R.as64(x), R.values(w), experts.cpu().numpy())
        assert (np.abs(R.as64(out) - want) <= R.matvec_adds(512, group) * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", GROUPS)
def test_rows_with_an_infinity_or_nan_give_nan_and_no_others(group, zero_points):
    w = make(2, 32, 512, group, zero_points)
    w.scale[0, 0, 3] = 0  # a row of weights whose first window is 0
    x = normal((11, 512), 3, dtype=torch.bfloat16)
    x[4, 77], x[5, 300], x[6, 511], x[7, 0] = float("nan"), float("inf"), -float("inf"), float("inf")
    x[7, 1] = -float("inf")
    bad, rest = [4, 5, 6, 7], [0, 1, 2, 3, 8, 9, 10]
    experts = torch.tensor([[0, 1]] * 11, dtype=torch.int32, device=DEV)
    weights = normal((11, 2), 4)
    clean = torch.where(x.isfinite(), x, 1.0)
    for more in (dict(), dict(act="silu"), dict(weights=weights)):
        for repeat in (1, 5):  # few rows and many
            call = {k: v if k == "act" else v.repeat(repeat, 1) for k, v in more.items()}
            args = (w, experts.repeat(repeat, 1))
            out = G.matvec_int4(x.repeat(repeat, 1), *args, **call, out_dtype=torch.float32)
            good = G.matvec_int4(clean.repeat(repeat, 1), *args, **call, out_dtype=torch.float32)
            for r in range(repeat):
                assert out[[11 * r + i for i in bad]].isnan().all()
                assert torch.equal(out[[11 * r + i for i in rest]], good[[11 * r + i for i in rest]])


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("power", [-120, -60, 60, 110])
def test_rows_of_any_size_with_and_without_zero_points(power, zero_points):
    w = make(3, 48, 768, 64, zero_points)
    x = normal((10, 768), 3, dtype=torch.bfloat16)
    x[2:5] *= 2.0 ** power
    x[6, 1:] = 0
    x[7] = 0
    experts = choose(10, 3, 2, 1, 0.0)
    for t in range(10):  # each row by its own size
        near(G.matvec_int4(x, w, experts, out_dtype=torch.float32)[t:t + 1], x[t:t + 1], w, experts[t:t + 1])
    assert not G.matvec_int4(x, w, experts, out_dtype=torch.float32)[7].any()
