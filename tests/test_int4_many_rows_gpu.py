"""Weights in 4-bit integers with the sorted rows of many tokens: gmm() takes the codes of groups of 128 without zero
points as they are, and any others dequantised.

Bounds.  Products of bf16 rows with whole numbers up to 8 and a scale for each 128 k are exact up to fp32 sums of k
terms, in any order, as matvec_int4()'s are: k units of 2^-23 of sum |w x|, and half a step of the output.
Dequantised weights have a rounding to bf16 of their own, half a step of each."""

import numpy as np
import pytest
import torch

import experts_reference as R
import moe_grouped_matrix_gb300 as G
from test_int4_gpu import DEV, choose, normal

pytestmark = pytest.mark.gpu


def scales_for_gmm(w):
    k = 2 * w.codes.shape[-1]
    return w.scale.transpose(2, 3).flatten(1, 2)[:, :k // 128, None].float().contiguous()


@pytest.mark.parametrize("tokens,experts,topk,n,k", [(5, 4, 2, 256, 256), (70, 6, 2, 384, 640), (300, 8, 2, 512, 1152),
                                                     (17, 16, 4, 136, 128)])
def test_gmm_takes_the_codes_and_their_scales(tokens, experts, topk, n, k):
    w = G.quantize_int4(normal((experts, n, k), 1, 0.05), 128)
    x, chosen = normal((tokens, k), 2, dtype=torch.bfloat16), choose(tokens, experts, topk, 3, 0.0)
    order = G.sort_by_expert(chosen, experts)
    rows, scales = G.dispatch(x, order), scales_for_gmm(w)
    assert scales.shape == (experts, k // 128, 1, n)
    got = G.gmm(rows, w.codes, order.group_sizes, scales, rhs_format="int4", out_dtype=torch.float32)
    back = G.gmm(rows, G.dequantize_int4(w), order.group_sizes, out_dtype=torch.float32)
    want, size = R.matvec(R.as64(x), R.values(w), chosen.cpu().numpy())
    at = order.rows.cpu().numpy()
    tol = k * 2.0 ** -23 * size + R.half_step(torch.float32) * np.abs(want)
    assert (np.abs(R.as64(got)[at] - want) <= tol).all()
    assert (np.abs(R.as64(back)[at] - want) <= tol + R.half_step(torch.bfloat16) * size).all()
    few = G.matvec_int4(x, w, chosen, out_dtype=torch.float32)
    assert (np.abs(R.as64(few) - R.as64(got)[at]) <= 2 * tol).all()


@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("group", [32, 64])
def test_other_groups_go_dequantised(group, zero_points):
    w = G.quantize_int4(normal((5, 264, 320), 1, 0.05), group, zero_points)
    x, chosen = normal((90, 320), 2, dtype=torch.bfloat16), choose(90, 5, 2, 3, 0.0)
    order = G.sort_by_expert(chosen, 5)
    got = G.gmm(G.dispatch(x, order), G.dequantize_int4(w), order.group_sizes, out_dtype=torch.float32)
    want, size = R.matvec(R.as64(x), R.values(w), chosen.cpu().numpy())
    tol = (320 * 2.0 ** -23 + R.half_step(torch.bfloat16)) * size
    assert (np.abs(R.as64(got)[order.rows.cpu().numpy()] - want) <= tol).all()
