"""balance_loss() and its gradient against the 64-bit statement.

Bounds, in units u = 2^-24.  A probability is a quotient of fp32 exponentials: l - max is off by |l - max| u at
most, the exponential, log sigmoid and the quotient by a few units, a sum of up to 1024 over a warp's tree by less
than 40: (64 + 4 max|l|) u of it.  Sums of T tokens, whatever their order, add T units, those over E experts E.
lse is a sum of two terms: (64 + 4 max|l|) u absolutely, and |lse| u.  A gradient's terms have the probabilities'
relative error; bf16 adds half a step."""

import numpy as np
import pytest
import torch

import experts_reference as R
import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(tokens, experts, topk, dtype, seed, dropped=0.1, off=0.1, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn((tokens, experts), generator=gen)).to(dtype)
    logits[torch.rand((tokens, experts), generator=gen) < off] = -float("inf")
    chosen = torch.randint(0, experts, (tokens, topk), generator=gen, dtype=torch.int32)
    chosen[torch.rand((tokens, topk), generator=gen) < dropped] = -1
    return logits, chosen


def check(logits, chosen, score="softmax", mask=None, sequences=1, pitch=0, dlosses=(0.7, -0.3)):
    T, E = logits.shape
    dl = logits.to(DEV)
    if pitch:
        wide = torch.full((T, E + pitch), float("nan"), dtype=logits.dtype, device=DEV)
        wide[:, :E] = dl
        dl = wide[:, :E]
    dm = None if mask is None else mask.to(DEV)
    b = G.balance_loss(dl, chosen.to(DEV), score, dm, sequences)
    d = torch.tensor(dlosses, dtype=torch.float32, device=DEV)
    g = G.balance_loss_backward(d, b, dl, score, dm)
    torch.cuda.synchronize()
    l64 = R.as64(logits)
    losses, counts, N, parts = R.balance(l64, chosen.numpy(), score, None if mask is None else mask.numpy(), sequences)
    assert b.losses.dtype == torch.float32 and b.counts.dtype == torch.int32 and g.dtype == logits.dtype
    np.testing.assert_array_equal(b.counts.cpu().numpy(), counts)
    assert b.tokens.tolist() == [N]
    live, p, f, lse, soft = parts
    top = np.abs(l64[live][np.isfinite(l64[live])]).max(initial=0.0)
    rel = (64 + 4 * top) * R.U32
    off = rel + np.abs(lse[live]) * R.U32
    z = ((2 * np.abs(lse[live]) + off) * off).sum() / max(N, 1) + (T + 8) * R.U32 * losses[1]
    got = R.as64(b.losses)
    assert abs(got[0] - losses[0]) <= (rel + (T + E + 8) * R.U32) * losses[0]
    assert abs(got[1] - losses[1]) <= z
    want, size = R.balance_gradient(R.as64(d), l64, parts, N, score)
    tol = (rel + (E + 16) * R.U32) * size + (R.half_step(logits.dtype) + R.U32) * np.abs(want) + 1e-38
    if logits.dtype == torch.bfloat16:
        tol += tol * 2.0 ** -8
    assert (np.abs(R.as64(g) - want) <= tol).all()
    return b, g


SHAPES = [(1, 1, 1, 1), (1, 8, 2, 1), (7, 3, 2, 1), (64, 64, 4, 2), (33, 61, 5, 3), (256, 128, 8, 16), (9, 160, 6, 9),
          (5, 257, 32, 1), (3, 1024, 32, 1), (4, 1000, 7, 2), (1500, 32, 2, 3), (2111, 250, 8, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_losses_loads_and_gradient(shape, dtype, score):
    tokens, experts, topk, sequences = shape
    logits, chosen = make(tokens, experts, topk, dtype, tokens + experts)
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(5)) > 0.2
    check(logits, chosen, score, None, sequences)
    bad = logits.clone()
    bad[~mask] = float("nan")  # not read into any result
    check(bad, chosen, score, mask, sequences, pitch=3)
    check(bad, chosen, score, mask.to(torch.uint8) * 7, sequences, pitch=8)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_sequences_and_one_large(score):
    logits, chosen = make(6000, 24, 3, torch.bfloat16, 11)
    for sequences in (1, 6000, 750):
        check(logits, chosen, score, None, sequences)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_that_do_not_count(score):
    logits, chosen = make(40, 12, 2, torch.float32, 3)
    logits[5] = -float("inf")        # its slots do not count either
    logits[6] = torch.finfo(torch.float32).min
    logits[6, 3] = 1.0
    logits[7, 1:] = -float("inf")    # one expert left
    chosen[5] = torch.tensor([1, 2])
    chosen[8] = torch.tensor([4, 4])  # the same expert twice
    chosen[9] = torch.tensor([12, -7])  # outside: dropped
    check(logits, chosen, score, None, 4)
    none = torch.zeros(40, dtype=torch.bool)
    b, g = check(logits, chosen, score, none, 4)  # a batch that is all padding
    assert b.losses.tolist() == [0.0, 0.0] and not g.any()
    none[3] = True
    check(logits, chosen, score, none, 4)
    check(logits, torch.full_like(chosen, -1), score, None, 2)  # every slot dropped


def test_no_tokens():
    b = G.balance_loss(torch.empty((0, 8), device=DEV), torch.empty((0, 2), dtype=torch.int32, device=DEV), sequences=3)
    g = G.balance_loss_backward(torch.ones(2, device=DEV), b, torch.empty((0, 8), device=DEV))
    assert b.losses.tolist() == [0.0, 0.0] and not b.counts.any() and b.counts.shape == (3, 8) and g.shape == (0, 8)


def test_large_and_tiny_logits():
    logits, chosen = make(64, 16, 2, torch.float32, 9, off=0.0)
    check(logits * 60, chosen, "softmax")
    check(logits * 60 - 300, chosen, "sigmoid")  # scores that fp32 has no number for
    check(logits * 1e-30, chosen, "sigmoid")


def test_a_nan_is_seen():
    logits, chosen = make(64, 16, 2, torch.float32, 9, off=0.0)
    logits[3, 4] = float("nan")
    b = G.balance_loss(logits.to(DEV), chosen.to(DEV))
    g = G.balance_loss_backward(torch.ones(2, device=DEV), b, logits.to(DEV))
    assert b.losses.isnan().all() and g[3].isnan().all() and not g[4:].isnan().any()


def test_equal_loads_give_one():
    logits = torch.randn((64, 8), device=DEV)
    chosen = (torch.arange(128, dtype=torch.int32, device=DEV) % 8).reshape(64, 2)
    b = G.balance_loss(logits, chosen)
    assert abs(float(b.losses[0]) - 1.0) < 100 * R.U32 and (b.counts == 16).all()


def test_the_same_bits_again():
    logits, chosen = make(5000, 128, 8, torch.bfloat16, 1)
    logits, chosen = logits.to(DEV), chosen.to(DEV)
    first = G.balance_loss(logits, chosen, sequences=5)
    for _ in range(20):
        assert torch.equal(first.losses, G.balance_loss(logits, chosen, sequences=5).losses)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """Central differences of the 64-bit losses with the loads held, whose own error is h^2 / 6 times a third
    derivative, of the size of the terms, and 2^-52 / h of the losses (of some 10)."""
    logits, chosen = make(12, 6, 2, torch.float32, 4, off=0.0)
    b = G.balance_loss(logits.to(DEV), chosen.to(DEV), score)
    d = torch.tensor([0.9, 0.2], device=DEV)
    got = R.as64(G.balance_loss_backward(d, b, logits.to(DEV), score))
    l, h, c = R.as64(logits), 1e-4, R.as64(d)
    for t in range(12):
        for e in range(6):
            hi, lo = l.copy(), l.copy()
            hi[t, e] += h
            lo[t, e] -= h
            diff = sum(c[i] * (R.balance(hi, chosen.numpy(), score)[0][i] - R.balance(lo, chosen.numpy(), score)[0][i])
                       for i in range(2)) / (2 * h)
            assert abs(got[t, e] - diff) < 1e-6


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_with_the_router(score):
    """route(), the losses of its choice and both gradients, as a training step adds them."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.randn((500, 32), generator=gen, device=DEV).to(torch.bfloat16)
    mask = torch.rand(500, generator=gen, device=DEV) > 0.1
    weights, experts = G.route(logits, 4, score, token_mask=mask)
    b, g = check(logits.cpu(), experts.cpu(), score, mask.cpu(), 2)
    assert int(b.counts.sum()) == 4 * int(mask.sum())
    assert torch.equal(b.counts.sum(0).to(torch.int32), G.sort_by_expert(experts, 32).group_sizes)
    total = g + G.route_backward(torch.ones_like(weights), experts, logits, score)
    assert total.isfinite().all() and not total[~mask].any()
