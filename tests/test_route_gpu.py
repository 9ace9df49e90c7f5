"""route() and route_backward() against the 64-bit statement.

Bounds.  A weight is a quotient of fp32 exponentials: the argument l - max carries a rounding of
at most 2^-24 |l - max|, the exponential and the logarithms a few units, a sum of up to 1024 terms
over a warp's tree less than 40 units, so (64 + 4 max|l|) * 2^-24 of the weight bounds it.  A
gradient is w (g - mean): the same relative error of |w| (|g| + mean |g|), which for all of a
token's experts is at most that of its sum of |g|, and half a unit of the output's format."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G
import moe_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(tokens, experts, dtype, seed, off=0.1, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn((tokens, experts), generator=gen)).to(dtype)
    logits[torch.rand((tokens, experts), generator=gen) < off] = -float("inf")
    return logits


def as64(t):
    return t.detach().cpu().double().numpy()


def relative(logits):
    l = as64(logits)
    return (64 + 4 * np.abs(l[np.isfinite(l)], where=True).max(initial=0.0)) * R.U32


def check_route(logits, topk, score, renormalize, scale=1.0, bias=None, mask=None):
    w, e = G.route(logits, topk, score, renormalize, scale, bias, mask)
    torch.cuda.synchronize()
    l32 = logits.detach().cpu().float().numpy()
    want = R.choose(l32, topk, None if bias is None else bias.cpu().numpy(), None if mask is None else mask.cpu().numpy())
    assert e.dtype == torch.int32 and w.dtype == torch.float32
    np.testing.assert_array_equal(e.cpu().numpy(), want)
    ref = R.weights_of(as64(logits), want, score, renormalize, scale)
    np.testing.assert_allclose(as64(w), ref, rtol=relative(logits), atol=1e-37)
    return w, e, ref


SHAPES = [(1, 8, 1), (1, 1, 1), (7, 8, 2), (64, 64, 4), (33, 61, 5), (130, 128, 8), (9, 160, 6), (5, 257, 32),
          (3, 1024, 32), (2, 1000, 7), (1031, 32, 32)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_choice_weights_and_gradient(shape, dtype, renormalize, score):
    tokens, experts, topk = shape
    logits = make(tokens, experts, dtype, tokens + experts).to(DEV)
    gen = torch.Generator().manual_seed(3)
    bias = (0.3 * torch.randn(experts, generator=gen)).to(DEV)
    mask = (torch.rand(tokens, generator=gen) > 0.2).to(DEV)
    logits[~mask] = float("nan")
    _, e, _ = check_route(logits, topk, score, renormalize, 2.5, bias, mask)
    g = torch.randn((tokens, topk), generator=gen).to(DEV)
    g[e < 0] = float("nan")  # slots without an expert do not count
    d = G.route_backward(g, e, logits, score, renormalize, 2.5)
    torch.cuda.synchronize()
    g64 = np.nan_to_num(as64(g))
    ref = R.route_gradient(g64, e.cpu().numpy(), as64(logits), score, renormalize, 2.5)
    assert d.dtype == logits.dtype
    unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    bound = relative(logits) * 2.5 * np.abs(g64).sum(1, keepdims=True) + unit * np.abs(ref) + 1e-37
    assert (np.abs(as64(d) - ref) <= bound).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(score, renormalize):
    """Central differences of the 64-bit weights: h^2 / 6 of a third derivative (below 6 for these
    functions, |g| <= 4) and 2^-52 / h of rounding are under 1e-6 at h = 2^-11."""
    logits = make(12, 40, torch.float32, 5, off=0.0)
    w, e = G.route(logits.to(DEV), 4, score, renormalize)
    g = torch.randn((12, 4), generator=torch.Generator().manual_seed(6)).clamp_(-4, 4)
    d = as64(G.route_backward(g.to(DEV), e, logits.to(DEV), score, renormalize))
    experts, l, h = e.cpu().numpy(), as64(logits), 2.0 ** -11
    for c in range(40):
        step = np.zeros_like(l)
        step[:, c] = h
        up = R.weights_of(l + step, experts, score, renormalize, 1.0)
        down = R.weights_of(l - step, experts, score, renormalize, 1.0)
        num = ((up - down) * as64(g)).sum(1) / (2 * h)
        assert np.abs(num - d[:, c]).max() < 16 * h * h + 16 * relative(logits)


def test_equal_keys_go_to_the_lowest_index():
    logits = torch.zeros((5, 200), device=DEV)
    logits[1, 100:] = 1.0
    logits[2, ::2] = -0.0
    logits[3, 7] = logits[3, 150] = 3.0
    _, e, _ = check_route(logits, 4, "softmax", True)
    assert e[0].tolist() == [0, 1, 2, 3] and e[1].tolist() == [100, 101, 102, 103]
    assert e[2].tolist() == [0, 1, 2, 3] and e[3].tolist() == [7, 150, 0, 1]


def test_rows_that_leave_nothing():
    inf = float("inf")
    logits = torch.full((4, 16), -inf, device=DEV)
    logits[1, 3] = -5.0  # one expert can be chosen
    logits[2] = torch.finfo(torch.float32).min  # the lowest finite value is no switch
    logits[3, 2], logits[3, 5] = float("nan"), 1.0
    for renormalize in (False, True):
        w, e = G.route(logits, 3, renormalize=renormalize)
        assert e[0].tolist() == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
        assert e[1].tolist() == [3, -1, -1] and w[1].tolist() == [1, 0, 0]
        assert e[2].tolist() == [0, 1, 2]
        assert torch.allclose(w[2], torch.full((3,), 1 / 3 if renormalize else 1 / 16, device=DEV))
        assert e[3].tolist() == [5, -1, -1]
    d = G.route_backward(torch.ones((4, 3), device=DEV), e, logits)
    assert d[0].abs().max() == 0 and d[1].abs().max() == 0


def test_large_logits_neither_overflow_nor_vanish():
    logits = torch.tensor([[300.0, 200.0, -300.0, 299.0], [-300.0, -301.0, -400.0, -500.0]], device=DEV)
    for score in ("softmax", "sigmoid"):
        check_route(logits, 2, score, True)
    w, _ = G.route(logits, 2, "sigmoid", True)
    assert torch.isfinite(w).all() and (w.sum(1) - 1).abs().max() < 1e-6


def test_rows_with_a_pitch_and_odd_addresses():
    for dtype in (torch.float32, torch.bfloat16):
        big = make(50, 300, dtype, 9).to(DEV)
        for lo, hi in ((0, 128), (1, 129), (8, 72), (3, 40)):
            view = big[:, lo:hi]
            w, e = G.route(view, 4)
            w2, e2 = G.route(view.contiguous(), 4)
            assert torch.equal(w, w2) and torch.equal(e, e2)
            g = torch.ones_like(w)
            assert torch.equal(G.route_backward(g, e, view, renormalize=False),
                               G.route_backward(g, e, view.contiguous(), renormalize=False))


def test_another_stream_and_a_graph():
    logits = make(64, 64, torch.float32, 11).to(DEV)
    want = G.route(logits, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = G.route(logits, 4)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = G.route(logits, 4)
    logits.copy_(make(64, 64, torch.float32, 12))
    graph.replay()
    torch.cuda.synchronize()
    want = G.route(logits, 4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens():
    w, e = G.route(torch.empty((0, 8), device=DEV), 2)
    assert w.shape == (0, 2) and e.shape == (0, 2)
    assert G.route_backward(w, e, torch.empty((0, 8), device=DEV)).shape == (0, 8)


def test_refusals():
    l = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError, match="topk"):
        G.route(l, 9)
    with pytest.raises(ValueError, match="topk"):
        G.route(l, 0)
    with pytest.raises(ValueError, match="score"):
        G.route(l, 2, score="tanh")
    with pytest.raises(TypeError):
        G.route(l.half(), 2)
    with pytest.raises(ValueError, match="dense rows"):
        G.route(l.t(), 2)
    with pytest.raises(ValueError, match="select_bias"):
        G.route(l, 2, select_bias=torch.zeros(7, device=DEV))
    with pytest.raises(TypeError, match="token_mask"):
        G.route(l, 2, token_mask=torch.zeros(4, device=DEV))
    with pytest.raises(G.GmmError, match="unsupported sizes"):
        G.route(torch.zeros((2, 1025), device=DEV), 2)
    w, e = G.route(l, 2)
    with pytest.raises(TypeError, match="experts"):
        G.route_backward(w, e.long(), l)
    with pytest.raises(ValueError, match="dweights"):
        G.route_backward(w[:2], e, l)
