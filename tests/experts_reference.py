"""Plain 64-bit statements of the router's balance, the gated activation, weights in 4-bit integers and
their products with few tokens, in numpy."""

import math

import numpy as np
import torch

U32 = 2.0 ** -24  # half the spacing of fp32 at 1
WINDOW = 256


def as64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- balance
def softmax(l):
    with np.errstate(invalid="ignore"):
        e = np.exp(l - l.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def balance(logits, experts, score="softmax", mask=None, sequences=1):
    """(losses [2], counts [S, E], N, and of each token: whether it counts, its p, f, lse and softmax)."""
    T, E = logits.shape
    live = np.ones(T, bool) if mask is None else mask.astype(bool).copy()
    live &= (logits != -np.inf).any(1)
    seq = np.arange(T) // (T // sequences) if T else np.zeros(0, int)
    counts = np.zeros((sequences, E), np.int64)
    for t in np.nonzero(live)[0]:
        for e in experts[t]:
            if 0 <= e < E:
                counts[seq[t], e] += 1
    l = np.where(live[:, None], logits, 0.0)
    soft = softmax(l)
    high = l.max(1)
    with np.errstate(invalid="ignore"):
        lse = high + np.log(np.exp(l - high[:, None]).sum(1))
    if score == "sigmoid":
        p = softmax(np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l))))
    else:
        p = soft
    f = (counts / np.maximum(counts.sum(1, keepdims=True), 1))[seq]
    N = int(live.sum())
    mean = (f * p).sum(1)
    losses = np.array([E * mean[live].sum(), (lse[live] ** 2).sum()]) / max(N, 1)
    return losses, counts, N, (live, p, f, lse, soft)


def balance_gradient(dlosses, logits, parts, N, score):
    """dlogits, and the sum of the sizes of its terms."""
    live, p, f, lse, soft = parts
    E = logits.shape[1]
    l = np.where(live[:, None], logits, 0.0)
    mean = (f * p).sum(1, keepdims=True)
    off = 1.0 / (1.0 + np.exp(l)) if score == "sigmoid" else 1.0
    a = dlosses[0] * E / max(N, 1) * p * off
    b = dlosses[1] * 2.0 / max(N, 1) * lse[:, None] * soft
    of = live[:, None]
    return (np.where(of, a * (f - mean) + b, 0.0),
            np.where(of, np.abs(a) * (f + mean)
                     + np.abs(dlosses[1] * 2.0 / max(N, 1) * soft) * (np.abs(lse) + 1)[:, None], 0.0))


# ---------------------------------------------------------------- the activation
def act(g, kind):
    """act(g), its slope, the argument x of g / (1 + exp(-x)), and the size of the slope's terms."""
    if kind == "silu":
        x, dx = g, np.ones_like(g)
    else:
        root = 2.0 * math.sqrt(2.0 / math.pi)
        x, dx = root * (g + 0.044715 * g ** 3), root * (1.0 + 3 * 0.044715 * g ** 2)
    e = np.exp(-np.abs(x))
    s = np.where(x < 0, e, 1.0) / (1.0 + e)
    rest = e / (1.0 + e) ** 2
    return g * s, s + g * rest * dx, x, s + np.abs(g) * rest * dx


# ---------------------------------------------------------------- 4-bit integers
def to_bf16(a):
    """fp32 values rounded to bf16, as 64-bit ones."""
    return torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).to(torch.bfloat16).double().numpy()


def quantize_int4(x, group, zero_points):
    """x [.., k] of 64-bit values that fp32 holds: codes, scales (64-bit), zero points (or None)."""
    g = x.reshape(x.shape[:-1] + (-1, group))
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    if zero_points:
        lo, hi = np.minimum(g.min(-1), 0.0), np.maximum(g.max(-1), 0.0)
        with np.errstate(over="ignore"):
            span = (hi - lo).astype(np.float32)
        fine &= np.isfinite(span)
        span = np.where(fine, span, 0).astype(np.float32)
        scale = to_bf16(span / np.float32(15))
    else:
        scale = to_bf16(np.abs(g).max(-1).astype(np.float32) / np.float32(7))
    safe = np.where(scale > 0, scale, 1.0)
    q = np.round(g / safe[..., None])  # quotients of 64 bits: exact where they lie half way
    zero = None
    if zero_points:
        zero = np.where(scale > 0, np.clip(np.round(-lo / safe), 0, 15), 0)
        q = np.clip(q + zero[..., None], 0, 15)
    else:
        q = np.clip(q, -8, 7)
    q = np.where((scale > 0)[..., None] & fine[..., None], q, 0)
    scale = np.where(fine, scale, np.nan)
    if zero is not None:
        zero = np.where(fine, zero, 0)
    return q.reshape(x.shape), scale, zero


def unpack(q):
    """codes, scales and zero points [.., rows, k / group] of an Int4Tensor, as 64-bit values."""
    codes = q.codes.cpu().numpy().astype(np.int64)
    k = 2 * codes.shape[-1]
    both = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (k,))

    def rows(t):
        a = as64(t) if t.dtype != torch.uint8 else t.cpu().numpy().astype(np.float64)
        a = np.moveaxis(a, -3, -2)
        return a.reshape(a.shape[:-2] + (-1,))[..., : k // q.group]

    if q.zero is None:
        both = (both + 8) % 16 - 8
    return both.astype(np.float64), rows(q.scale), None if q.zero is None else rows(q.zero)


def values(q):
    codes, scale, zero = unpack(q)
    v = codes.reshape(codes.shape[:-1] + (-1, q.group))
    if zero is not None:
        v = v - zero[..., None]
    return (v * scale[..., None]).reshape(codes.shape)


def term_sizes(q):
    """Of the terms scale code x and scale zero x, codes counted from 0: what multiplies |x|."""
    codes, scale, zero = unpack(q)
    v = codes.reshape(codes.shape[:-1] + (-1, q.group))
    v = v + 16.0 if zero is None else v + zero[..., None]  # (code + 8) + 8
    return (v * scale[..., None]).reshape(codes.shape)


def matvec(x, w, experts, weights=None, kind=None, sizes=None):
    """(out, size of the terms of each sum): x [T, k] or [T, K, k], w [E, n, k], all 64-bit; the terms are
    |w x|, or those of term_sizes()."""
    sizes = np.abs(w) if sizes is None else sizes
    T, K = experts.shape
    n = w.shape[1]
    h, size = np.zeros((T, K, n)), np.zeros((T, K, n))
    for t in range(T):
        for j in range(K):
            e = experts[t, j]
            if 0 <= e < w.shape[0]:
                v = x[t, j] if x.ndim == 3 else x[t]
                h[t, j], size[t, j] = w[e] @ v, sizes[e] @ np.abs(v)
    if kind is not None:
        f = n // 2
        a, slope, arg, slopes = act(h[..., :f], kind)
        u = h[..., f:]
        # what an error of `size` units in either half moves the product by, and the activation's own
        own = (16 + 8 * np.abs(arg)) * np.abs(a * u)
        size = np.abs(slope) * size[..., :f] * np.abs(u) + np.abs(a) * size[..., f:] + own
        h = a * u
    if weights is not None:
        h, size = (h * weights[..., None]).sum(1), (size * np.abs(weights)[..., None]).sum(1)
    return h, size


def matvec_adds(k, group):
    """Roundings that a sum's term goes through, in units of 2^-23 (the matrix instructions may cut off):
    16 products and the sum so far in each of a group's instructions (or the sum of x that the zero point takes),
    then the groups, the warps, the slots."""
    return 2 * (group // 16) + -(-k // group) + 8 + 32
