"""sort_by_expert(), dispatch(), combine() and their gradients against the 64-bit statement.

Bounds.  The order and dispatch() are exact.  combine() is a chain of topk fused multiply-adds in
fp32: at most topk * 2^-24 of the sum of magnitudes, and half a unit of the output's format.  A
gradient row is one product rounded once.  dweights are fp32 dot products of d terms: at most
(d + 8) * 2^-24 of the sum of magnitudes in any order."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G
import moe_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


def as64(t):
    return t.detach().cpu().double().numpy()


def choice(tokens, topk, experts, seed, dropped=0.0):
    gen = torch.Generator().manual_seed(seed)
    e = torch.argsort(torch.rand((tokens, max(experts, topk)), generator=gen), dim=1)[:, :topk] % experts
    e = (e * e // experts).to(torch.int32)  # uneven
    e[torch.rand((tokens, topk), generator=gen) < dropped] = -1
    return e


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 4, 64), (64, 4, 64), (1000, 3, 7), (4096, 1, 1024),
                                                 (4097, 1, 5), (1025, 4, 128), (5000, 8, 128), (33000, 8, 1024),
                                                 (20011, 32, 3)])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_order(tokens, topk, experts, dropped):
    e = choice(tokens, topk, experts, tokens, dropped)
    if dropped:
        e[::5] = experts  # outside the range: dropped too
    order = G.sort_by_expert(e.to(DEV), experts)
    torch.cuda.synchronize()
    sizes, rows, source = R.order_of(e.numpy(), experts)
    np.testing.assert_array_equal(order.group_sizes.cpu().numpy(), sizes)
    np.testing.assert_array_equal(order.rows.cpu().numpy(), rows)
    np.testing.assert_array_equal(order.source.cpu().numpy(), source)


def test_any_int32_is_an_expert_or_dropped():
    e = torch.tensor([[2 ** 31 - 1, -2 ** 31, 0], [3, 4, -1]], dtype=torch.int32)
    order = G.sort_by_expert(e.to(DEV), 4)
    assert order.group_sizes.tolist() == [1, 0, 0, 1]
    assert order.rows.tolist() == [[-1, -1, 0], [1, -1, -1]]
    assert order.source.tolist() == [2, 3, -1, -1, -1, -1]


SHAPES = [(1, 1, 1, 1), (1, 4, 64, 4096), (64, 4, 64, 2048), (37, 3, 9, 1027), (100, 5, 16, 33), (50, 8, 128, 1000),
          (513, 2, 8, 4100), (9, 32, 40, 66), (3, 2, 4, 40000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dropped", [0.0, 0.2, 1.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_there_and_back(shape, dropped, dtype):
    tokens, topk, experts, d = shape
    e = choice(tokens, topk, experts, 5, dropped)
    order = G.sort_by_expert(e.to(DEV), experts)
    sizes, rows_of, source = R.order_of(e.numpy(), experts)
    gen = torch.Generator().manual_seed(7)
    x = torch.randn((tokens, d), generator=gen).to(dtype).to(DEV)
    got = G.dispatch(x, order)
    want = np.zeros((tokens * topk, d))
    want[source >= 0] = as64(x)[source[source >= 0] // topk]
    np.testing.assert_array_equal(as64(got), want)

    rows = torch.randn((tokens * topk, d), generator=gen).to(dtype).to(DEV)
    rows[torch.from_numpy(source < 0).to(DEV)] = float("nan")  # past the groups: nobody's
    w = torch.randn((tokens, topk), generator=gen).to(DEV)
    took = rows_of >= 0
    taken = np.where(took[..., None], as64(rows)[np.maximum(rows_of, 0)], 0.0)
    for weights in (w, None):
        out = G.combine(rows, order, weights)
        w64 = np.where(took, 1.0 if weights is None else as64(w), 0.0)
        ref = (taken * w64[..., None]).sum(1)
        mag = np.abs(taken * w64[..., None]).sum(1)
        assert out.dtype == dtype
        assert (np.abs(as64(out) - ref) <= topk * R.U32 * mag + UNIT[dtype] * np.abs(ref)).all()
    assert torch.equal(G.dispatch_backward(rows, order), G.combine(rows, order))

    dout = torch.randn((tokens, d), generator=gen).to(dtype).to(DEV)
    drows, dw = G.combine_backward(dout, rows, order, w)
    ref = np.zeros((tokens * topk, d))
    live = source >= 0
    ref[live] = as64(dout)[source[live] // topk] * as64(w).reshape(-1)[source[live]][:, None]
    assert drows.dtype == dtype and dw.dtype == torch.float32
    assert (np.abs(as64(drows) - ref) <= UNIT[dtype] * np.abs(ref)).all()
    terms = taken * as64(dout)[:, None, :]
    assert (np.abs(as64(dw) - terms.sum(2)) <= (d + 8) * R.U32 * np.abs(terms).sum(2)).all()
    again = G.combine_backward(dout, rows, order, w)
    assert torch.equal(drows, again[0]) and torch.equal(dw, again[1])


def test_gradients_against_differences():
    """combine() is linear in rows and in weights, and integers this small are exact: the
    difference quotient of <dout, combine> is the gradient itself."""
    tokens, topk, d = 6, 3, 20
    order = G.sort_by_expert(choice(tokens, topk, 5, 1, 0.2).to(DEV), 5)
    gen = torch.Generator().manual_seed(2)

    def ints(*shape):
        return torch.randint(-4, 5, shape, generator=gen).float().to(DEV)

    rows, w, dout = ints(tokens * topk, d), ints(tokens, topk), ints(tokens, d)
    drows, dw = G.combine_backward(dout, rows, order, w)
    base = (dout * G.combine(rows, order, w)).sum()
    for t in range(tokens):
        for j in range(topk):
            v = w.clone()
            v[t, j] += 1
            assert (dout * G.combine(rows, order, v)).sum() - base == dw[t, j]
    for r in range(0, tokens * topk):
        v = rows.clone()
        v[r, r] += 1
        assert (dout * G.combine(v, order, w)).sum() - base == drows[r, r]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_with_a_pitch_and_odd_addresses(dtype):
    order = G.sort_by_expert(choice(40, 2, 8, 3).to(DEV), 8)
    big = torch.randn((40, 600), device=DEV).to(dtype)
    for lo, hi in ((0, 512), (1, 513), (4, 260), (2, 33)):
        view = big[:, lo:hi]
        assert torch.equal(G.dispatch(view, order), G.dispatch(view.contiguous(), order))
    flat = torch.randn(80 * 64 + 1, device=DEV).to(dtype)
    odd = flat[1:].view(80, 64)
    w = torch.randn((40, 2), device=DEV)
    assert torch.equal(G.combine(odd, order, w), G.combine(odd.clone(), order, w))
    dout = torch.randn((40, 64), device=DEV).to(dtype)
    a, b = G.combine_backward(dout, odd, order, w), G.combine_backward(dout, odd.clone(), order, w)
    assert torch.equal(a[0], b[0])
    # the dot products are summed in another order: d + 8 roundings each way
    assert torch.allclose(a[1], b[1], rtol=0, atol=2 * 72 * 2.0 ** -24 * 64 * 16)


def test_infinities_stay_where_they_are():
    order = G.sort_by_expert(torch.tensor([[0, 1], [1, 0]], dtype=torch.int32, device=DEV), 2)
    rows = torch.ones((4, 8), device=DEV)
    rows[order.rows[0, 0], 3] = float("inf")
    out = G.combine(rows, order, torch.full((2, 2), 0.5, device=DEV))
    assert out[0, 3] == float("inf") and torch.isfinite(out).sum() == 15


def test_offsets_past_32_bits():
    tokens, topk, d = 75000, 8, 4096  # 2.46e9 elements of rows
    e = torch.randint(0, 16, (tokens, topk), dtype=torch.int32, device=DEV)
    order = G.sort_by_expert(e, 16)
    x = torch.randn((tokens, d), device=DEV).to(torch.bfloat16)
    rows = G.dispatch(x, order)
    at = torch.randint(0, tokens * topk, (2000,), device=DEV)
    at[0] = tokens * topk - 1
    assert torch.equal(rows[at], x[(order.source[at] // topk).long()])
    out = G.combine(rows, order)
    assert torch.equal(out, x * topk)
    w = torch.full((tokens, topk), 0.5, device=DEV)
    drows, dw = G.combine_backward(x, rows, order, w)
    assert torch.equal(drows[at], rows[at] * 0.5)
    assert torch.allclose(dw[:, 0], x.float().square().sum(1), rtol=1e-4)


def test_another_stream_and_a_graph():
    e = choice(300, 4, 16, 8).to(DEV)
    x = torch.randn((300, 256), device=DEV)
    w = torch.rand((300, 4), device=DEV)

    def there_and_back():
        order = G.sort_by_expert(e, 16)
        return G.combine(G.dispatch(x, order), order, w)

    want = there_and_back()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = there_and_back()
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = there_and_back()
    e.copy_(choice(300, 4, 16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, there_and_back())


def test_calls_that_follow_each_other_closely():
    """Each call reads what the one before wrote, through memory that the allocator hands out again and
    again: halves of two equal rows are the row itself, so nothing may change."""
    order = G.sort_by_expert(choice(500, 2, 16, 4).to(DEV), 16)
    x = torch.randn((500, 1024), device=DEV)
    half = torch.full((500, 2), 0.5, device=DEV)
    y = x
    for _ in range(500):
        y = G.combine(G.dispatch(y, order), order, half)
    assert torch.equal(y, x)


def test_no_tokens():
    order = G.sort_by_expert(torch.empty((0, 2), dtype=torch.int32, device=DEV), 4)
    assert order.group_sizes.tolist() == [0, 0, 0, 0]
    rows = G.dispatch(torch.empty((0, 8), device=DEV), order)
    assert rows.shape == (0, 8) and G.combine(rows, order).shape == (0, 8)
    a, b = G.combine_backward(torch.empty((0, 8), device=DEV), rows, order, torch.empty((0, 2), device=DEV))
    assert a.shape == (0, 8) and b.shape == (0, 2)


def test_refusals():
    e = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError, match="experts"):
        G.sort_by_expert(e.long(), 4)
    with pytest.raises(ValueError, match="experts"):
        G.sort_by_expert(e.view(-1), 4)
    with pytest.raises(G.GmmError, match="unsupported sizes"):
        G.sort_by_expert(e, 0)
    with pytest.raises(G.GmmError, match="unsupported sizes"):
        G.sort_by_expert(e, 1025)
    with pytest.raises(G.GmmError, match="unsupported sizes"):
        G.sort_by_expert(torch.zeros((1, 33), dtype=torch.int32, device=DEV), 4)
    order = G.sort_by_expert(e, 4)
    x = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError, match="4 rows"):
        G.dispatch(x[:3], order)
    with pytest.raises(TypeError):
        G.dispatch(x.half(), order)
    with pytest.raises(ValueError, match="dense rows"):
        G.dispatch(torch.zeros((8, 4), device=DEV).t(), order)
    rows = G.dispatch(x, order)
    with pytest.raises(ValueError, match="rows must be"):
        G.combine(rows[:7], order)
    with pytest.raises(ValueError, match="weights"):
        G.combine(rows, order, torch.zeros((4, 3), device=DEV))
    with pytest.raises(TypeError, match="dout"):
        G.combine_backward(x.bfloat16(), rows, order, torch.zeros((4, 2), device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        G.combine(torch.zeros((8, 16), device=DEV)[:, :8], order)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,topk,experts,d", [(7, 3, 4, 20001), (40, 8, 16, 7168), (300, 2, 8, 515),
                                                   (1216, 5, 8, 1026), (1217, 5, 8, 1027), (1300, 3, 8, 1028),
                                                   (1500, 2, 8, 2056), (2000, 1, 8, 64), (2500, 7, 8, 129)])
def test_gradients_of_few_and_of_many_tokens(tokens, topk, experts, d, dtype):
    """A gradient row is w * dout rounded once; dweights within their bound, 0 for a dropped slot."""
    e = choice(tokens, topk, experts, d, 0.1)
    order = G.sort_by_expert(e.to(DEV), experts)
    gen = torch.Generator(DEV).manual_seed(d)
    rows = torch.randn((tokens * topk, d), generator=gen, device=DEV).to(dtype)
    dout = torch.randn((tokens, d), generator=gen, device=DEV).to(dtype)
    w = torch.rand((tokens, topk), generator=gen, device=DEV)
    drows, dw = G.combine_backward(dout, rows, order, w)
    kept = order.rows >= 0
    want = torch.zeros_like(rows)
    want[order.rows[kept].long()] = (w[..., None] * dout.float()[:, None])[kept].to(dtype)
    assert torch.equal(drows, want)
    at = order.rows.long().clamp_min(0)
    for j in range(topk):
        prod = dout.double() * rows[at[:, j]].double() * kept[:, j, None]
        assert ((dw[:, j].double() - prod.sum(1)).abs() <= (d + 8) * 2.0 ** -24 * prod.abs().sum(1)).all()


@pytest.mark.parametrize("d", [64, 99, 1030])
def test_dropped_slots_have_no_gradient_whatever_dout_holds(d):
    e = torch.full((4, 3), -1, dtype=torch.int32)
    e[:, 1] = torch.tensor([0, 1, 1, 2])
    order = G.sort_by_expert(e.to(DEV), 3)
    rows = torch.ones((12, d), device=DEV)
    dout = torch.ones((4, d), device=DEV)
    dout[0, 0], dout[1, d - 1], dout[2, d // 2] = float("nan"), float("inf"), -float("inf")
    drows, dw = G.combine_backward(dout, rows, order, torch.ones((4, 3), device=DEV))
    assert (dw[:, [0, 2]] == 0).all()
    assert torch.equal(dw[1:, 1], torch.tensor([float("inf"), -float("inf"), float(d)], device=DEV))
    assert dw[0, 1].isnan() and (drows[4:] == 0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,topk,d,dtype", [(2048, 3, 2048, torch.bfloat16), (2047, 3, 2048, torch.bfloat16),
                                                 (2049, 1, 2056, torch.bfloat16), (6000, 5, 520, torch.float32),
                                                 (1025, 6, 2052, torch.float32)])
def test_sums_of_many_rows(tokens, topk, d, dtype, weighted):
    """Around the size from which combine() takes longer runs of a row: a token's sum is the same chain,
    to the bit, as in a call of few tokens."""
    e = choice(tokens, topk, 16, d, 0.1)
    order = G.sort_by_expert(e.to(DEV), 16)
    gen = torch.Generator(DEV).manual_seed(d)
    rows = torch.randn((tokens * topk, d), generator=gen, device=DEV).to(dtype)
    w = torch.rand((tokens, topk), generator=gen, device=DEV) if weighted else None
    got = G.combine(rows, order, w)
    for t0 in (0, tokens // 2, tokens - 100):
        few = G.sort_by_expert(e[t0:t0 + 100].to(DEV), 16)
        kept = few.rows >= 0
        part = torch.full((100 * topk, d), float("nan"), device=DEV, dtype=dtype)
        part[few.rows[kept].long()] = rows[order.rows[t0:t0 + 100][kept].long()]
        assert torch.equal(got[t0:t0 + 100], G.combine(part, few, w[t0:t0 + 100] if weighted else None))
