"""route() with a selection bias on the scores: the topk largest s(l) + b, s the softmax over all experts or
the sigmoid, against the 64-bit statement.

Bounds.  A score is a quotient of fp32 exponentials, its relative error at most (64 + 4 max|l|) * 2^-24 as
for the weights; the sum with the bias adds 2^-24 of itself.  So a key is known to d = that much, and the
choice is right if no chosen expert's exact key lies more than 2 d below one that should have come in its
place.  Where all neighbouring keys of a token are further apart than that, the choice is the exact one."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G
import moe_reference as R
from test_route_gpu import DEV, SHAPES, as64, make, relative

pytestmark = pytest.mark.gpu


def keys_of(logits, bias, score, mask):
    """Exact keys [T, E], -inf where an expert cannot be chosen, and what each is known to."""
    l = as64(logits)
    if mask is not None:
        l[~mask.cpu().numpy()] = -np.inf
    s = R._scores(np.where(np.isfinite(l).any(1, keepdims=True), l, 0.0), score)
    key = np.where(l > -np.inf, s + as64(bias), -np.inf)
    finite = np.where(np.isfinite(key), key, 0.0)
    return key, relative(logits) * s + R.U32 * np.abs(finite)


def check_choice(e, logits, topk, score, bias, mask=None):
    """e is the choice of the exact keys, up to what the keys are known to; the tokens decided exactly."""
    key, known = keys_of(logits, bias, score, mask)
    order = np.argsort(-key, axis=1, kind="stable")
    top = np.take_along_axis(key, order, 1)[:, :topk + 1]
    d = known.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        gaps = top[:, :-1] - top[:, 1:]
    clear = (np.nan_to_num(gaps, nan=np.inf) > 2 * d).all(1)
    want = np.where(top[:, :topk] > -np.inf, order[:, :topk], -1)
    got = e.cpu().numpy()
    np.testing.assert_array_equal(got[clear], want[clear])
    np.testing.assert_array_equal(got >= 0, want >= 0)
    for t in range(len(got)):
        mine = got[t][got[t] >= 0]
        assert len(set(mine)) == len(mine)
        assert (key[t, mine] >= top[t, :len(mine)] - 2 * d[t]).all()
    return clear


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_choice_weights_and_gradient(shape, dtype, renormalize, score):
    tokens, experts, topk = shape
    logits = make(tokens, experts, dtype, 2 * tokens + experts).to(DEV)
    gen = torch.Generator().manual_seed(4)
    bias = (0.3 * torch.randn(experts, generator=gen)).to(DEV)
    mask = (torch.rand(tokens, generator=gen) > 0.2).to(DEV)
    logits[~mask] = float("nan")
    w, e = G.route(logits, topk, score, renormalize, 2.5, bias, mask, bias_on="score")
    check_choice(e, logits, topk, score, bias, mask)
    chosen = e.cpu().numpy()
    ref = R.weights_of(as64(logits), chosen, score, renormalize, 2.5)
    np.testing.assert_allclose(as64(w), ref, rtol=relative(logits), atol=1e-37)
    g = torch.randn((tokens, topk), generator=gen).to(DEV)
    d = G.route_backward(g, e, logits, score, renormalize, 2.5)
    want = R.route_gradient(as64(g), chosen, as64(logits), score, renormalize, 2.5)
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    bound = relative(logits) * 2.5 * np.abs(as64(g)).sum(1, keepdims=True) + unit * np.abs(want) + 1e-37
    assert (np.abs(as64(d) - want) <= bound).all()


def test_most_tokens_are_decided_exactly():
    logits = make(2000, 64, torch.float32, 8).to(DEV)
    bias = (0.3 * torch.randn(64, generator=torch.Generator().manual_seed(5))).to(DEV)
    for score in ("softmax", "sigmoid"):
        _, e = G.route(logits, 4, score, select_bias=bias, bias_on="score")
        assert check_choice(e, logits, 4, score, bias).mean() > 0.99


def test_a_bias_on_the_score_chooses_others_than_one_on_the_logit():
    logits = torch.tensor([[4.0, 0.0, -1.0]], device=DEV)
    bias = torch.tensor([0.0, 0.6, 0.0], device=DEV)
    for short in (True, False):
        scale = 1.0 if short else 1
        w, e = G.route(logits, 1, "sigmoid", False, scale, bias)
        assert e.tolist() == [[0]]
        w, e = G.route(logits, 1, "sigmoid", False, scale, bias, bias_on="score")  # 0.982 against 0.5 + 0.6
        assert e.tolist() == [[1]] and w.tolist() == [[0.5]]  # the weight is the score's, without the bias


def test_equal_keys_go_to_the_lowest_index():
    logits = torch.full((3, 100), 0.7, device=DEV)
    logits[1, 60:] = 1.5
    bias = torch.zeros(100, device=DEV)
    bias[40:] = 0.125
    for score in ("softmax", "sigmoid"):
        _, e = G.route(logits, 3, score, select_bias=bias, bias_on="score")
        assert e.tolist() == [[40, 41, 42], [60, 61, 62], [40, 41, 42]]
        _, e = G.route(logits, 3, score, bias_on="score")  # without a bias the scores' order is the logits'
        assert e.tolist() == [[0, 1, 2], [60, 61, 62], [0, 1, 2]]


def test_rows_that_leave_nothing():
    inf, nan = float("inf"), float("nan")
    logits = torch.zeros((5, 8), device=DEV)
    logits[0] = -inf
    logits[1, 1:] = -inf
    logits[2, 3] = nan
    logits[3, 2] = inf
    logits[4] = torch.finfo(torch.float32).min  # the lowest finite value is no switch
    bias = torch.full((8,), 5.0, device=DEV)
    bias[6], bias[7] = -inf, nan  # never chosen
    w, e = G.route(logits, 2, "sigmoid", select_bias=bias, bias_on="score")
    assert e.tolist() == [[-1, -1], [0, -1], [0, 1], [2, 0], [0, 1]]
    assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0] and torch.isfinite(w).all()
    w, e = G.route(logits, 2, "softmax", select_bias=bias, bias_on="score")
    assert e.tolist() == [[-1, -1], [0, -1], [-1, -1], [-1, -1], [0, 1]]  # a row whose scores are NaN has no keys
    assert w[2].tolist() == [0, 0] and w[4].tolist() == [0.5, 0.5]


def test_large_logits_neither_overflow_nor_vanish():
    logits = torch.tensor([[300.0, 200.0, -300.0, 299.0]], device=DEV)
    bias = torch.tensor([0.0, 0.25, 1.5, 0.0], device=DEV)
    for score, want in (("softmax", [2, 0, 3]), ("sigmoid", [2, 1, 0])):
        _, e = G.route(logits, 3, score, select_bias=bias, bias_on="score")
        assert e[0].tolist() == want


def test_a_given_stream_and_refusals():
    logits = make(300, 24, torch.float32, 3).to(DEV)
    bias = torch.linspace(0, 1, 24, device=DEV)
    want = G.route(logits, 3, "sigmoid", select_bias=bias, bias_on="score")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = G.route(logits, 3, "sigmoid", select_bias=bias, stream=side, bias_on="score")
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for over in (dict(bias_on="weight"), dict(bias_on=None), dict(bias_on="weight", stream=side)):
        with pytest.raises(ValueError, match="bias_on"):
            G.route(logits, 3, select_bias=bias, **over)
    with pytest.raises(ValueError, match="score"):
        G.route(logits, 3, "tanh", select_bias=bias, bias_on="score")
