"""More operators of a mixture-of-experts layer, behind the C ABI of libgmm
(``include/libgmm_experts.h``): the losses that balance the router, the gated activation between an
expert's two products, weights in 4-bit integers with group scales, and their products with few tokens.

    b = balance_loss(logits, experts)              # b.losses [2]: balance and z; b.counts: the loads
    dlogits = balance_loss_backward(dlosses, b, logits)
    act = gated_act(h)                             # silu(first half) * second half
    w = quantize_int4(weights, group=128)          # once
    h = matvec_int4(x, w, experts, act="silu")     # [tokens, topk, n / 2], no sort
    y = matvec_int4(h, w2, experts, weights)       # [tokens, n], weighted and summed

Conventions are ``moe.py``'s: arguments are checked and marshalled here, gradients are calls of their
own, and a call with ``stream=`` runs there and its results belong to that stream.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _I, _I32, _I64, _P, _SZ, SIGNATURES, _dev, _on_stream
from . import moe as _moe
from .moe import _OUT_F32, MAX_TOPK, SCORES, _float_code, _lib, _on, _ptr, _rows, _run, _score, _want

__all__ = ["BalanceLoss", "balance_loss", "balance_loss_backward", "gated_act", "gated_act_backward", "Int4Tensor",
           "quantize_int4", "dequantize_int4", "matvec_int4"]

ACTS = {"silu": 1, "gelu": 2}
INT4_GROUPS = (32, 64, 128)
_WINDOW = 256

SIGNATURES.update({
    "gmm_balance_scratch_bytes": ([_I64, _I32, _I64], _SZ),
    "gmm_balance_loss": ([_P, _I, _I64, _I32, _I64, _P, _I32, _I, _P, _I64, _P, _P, _P, _P, _SZ, _P], _I),
    "gmm_balance_loss_backward": ([_P, _P, _P, _P, _I, _I64, _I32, _I64, _I, _P, _I64, _P, _P], _I),
    "gmm_gated_act": ([_P, _I, _I64, _I64, _I64, _I, _P, _P], _I),
    "gmm_gated_act_backward": ([_P, _P, _I, _I64, _I64, _I64, _I, _P, _P], _I),
    "gmm_quantize_int4": ([_P, _I, _I32, _I64, _I64, _I64, _I32, _P, _P, _P, _P], _I),
    "gmm_dequantize_int4": ([_P, _P, _P, _I32, _I32, _I64, _I64, _P, _I, _P], _I),
    "gmm_matvec_int4": ([_P, _I64, _I64, _I64, _I, _P, _P, _P, _I32, _I32, _I64, _P, _I32, _P, _I, _P, _I, _P, _SZ, _P],
                        _I),
    "gmm_matvec_scratch_bytes": ([_I64, _I64, _I32, _I, _I32, _I], _SZ),
})


class BalanceLoss(NamedTuple):
    """balance_loss()'s results: losses float32 [2] (the balance loss and the z loss, without
    coefficients), counts int32 [sequences, experts] (the slots each expert got), tokens int32 [1]
    (how many tokens counted)."""
    losses: torch.Tensor
    counts: torch.Tensor
    tokens: torch.Tensor


class Int4Tensor(NamedTuple):
    """Matrices [.., rows, k] of 4-bit integers: codes uint8 [.., rows, k / 2] (even k in the low
    nibble), scale bfloat16 [.., ceil(k / 256), rows, 256 / group] (a row's scales by windows of 256
    k), zero uint8 like scale, or None, and the group of k (32, 64 or 128) that shares a scale.  They
    stand for scale * code with two's complement codes, or with zero for scale * (code - zero), codes 0 to 15."""
    codes: torch.Tensor
    scale: torch.Tensor
    zero: Optional[torch.Tensor]
    group: int


def _token_mask(mask, tokens):
    if mask is not None:
        _want(mask, "token_mask", torch.uint8 if mask.dtype == torch.uint8 else torch.bool, (tokens,))


def balance_loss(logits, experts, score="softmax", token_mask=None, sequences=1, stream=None):
    """The losses that keep a router's experts evenly loaded, and the loads, as a BalanceLoss.  logits
    [tokens, E] (bfloat16 or float32, rows may have a pitch), experts int32 [tokens, topk] as route()
    chose them.  With p a token's softmax (or, score="sigmoid", its sigmoids over their sum) and f each
    expert's share of the slots of the token's sequence, the balance loss is E times the mean over
    tokens of <f, p>, and the z loss the mean of logsumexp(logits)^2.  The tokens are `sequences` runs
    of equal length, each with loads of its own.  Tokens whose token_mask (bool or uint8 [tokens]) is
    0, or whose logits are all -inf, do not count; slots outside [0, E) are dropped."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).balance_loss(logits, experts, SCORES.get(score), token_mask, sequences)
        if got.__class__ is tuple:
            return BalanceLoss._make(got)
        _run("gmm_balance_loss", got)
    ld = _rows(logits, "logits")
    code = _float_code(logits, "logits")
    tokens, n = logits.shape
    if experts.dim() != 2:
        raise ValueError("experts must be [tokens, topk]")
    topk = experts.shape[1]
    _want(experts, "experts", torch.int32, (tokens, topk))
    _token_mask(token_mask, tokens)
    sequences = int(sequences)
    if sequences < 1 or tokens % sequences:
        raise ValueError(f"sequences must divide {tokens} tokens")
    lib = _lib()
    nbytes = lib.gmm_balance_scratch_bytes(tokens, n, sequences)
    with _on_stream(stream):
        losses = torch.empty((2,), dtype=torch.float32, device=logits.device)
        counts = torch.empty((sequences, n), dtype=torch.int32, device=logits.device)
        counted = torch.empty((1,), dtype=torch.int32, device=logits.device)
        scratch = torch.empty((nbytes,), dtype=torch.uint8, device=logits.device) if nbytes else None
    _run("gmm_balance_loss", lib.gmm_balance_loss(
        logits.data_ptr(), code, tokens, n, ld, experts.data_ptr(), topk, _score(score), _ptr(token_mask), sequences,
        losses.data_ptr(), counts.data_ptr(), counted.data_ptr(), _ptr(scratch), nbytes,
        _on(logits.device, stream)))
    return BalanceLoss(losses, counts, counted)


def balance_loss_backward(dlosses, balance, logits, score="softmax", token_mask=None, stream=None):
    """Gradient of <dlosses, balance.losses> with respect to the logits, [tokens, E] of their dtype:
    dlosses float32 [2] (the losses' coefficients times the gradient they get), balance the
    BalanceLoss of these logits with the same score and token_mask."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).balance_loss_backward(dlosses, balance.counts, balance.tokens, logits,
                                                                  SCORES.get(score), token_mask)
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_balance_loss_backward", got)
    ld = _rows(logits, "logits")
    code = _float_code(logits, "logits")
    tokens, n = logits.shape
    if balance.counts.dim() != 2 or balance.counts.shape[0] < 1 or tokens % balance.counts.shape[0]:
        raise ValueError(f"balance.counts must be [sequences, {n}] with sequences that divide {tokens} tokens")
    sequences = balance.counts.shape[0]
    _want(balance.counts, "balance.counts", torch.int32, (sequences, n))
    _want(balance.tokens, "balance.tokens", torch.int32, (1,))
    _want(dlosses, "dlosses", torch.float32, (2,))
    _token_mask(token_mask, tokens)
    with _on_stream(stream):
        dlogits = torch.empty((tokens, n), dtype=logits.dtype, device=logits.device)
    _run("gmm_balance_loss_backward", _lib().gmm_balance_loss_backward(
        dlosses.data_ptr(), balance.counts.data_ptr(), balance.tokens.data_ptr(), logits.data_ptr(), code, tokens, n,
        ld, _score(score), _ptr(token_mask), sequences, dlogits.data_ptr(), _on(logits.device, stream)))
    return dlogits


def _act(act):
    try:
        return ACTS[act]
    except KeyError:
        raise ValueError(f"act must be one of {sorted(ACTS)}") from None


def _halves(h):
    ld = _rows(h, "h")
    if h.shape[1] % 2 or h.shape[1] == 0:
        raise ValueError("h must be [rows, 2 f]")
    return ld, h.shape[1] // 2


def gated_act(h, act="silu", stream=None):
    """act(h[:, :f]) * h[:, f:] in fp32, rounded once: [rows, f] from h [rows, 2 f] (bfloat16 or
    float32, rows may have a pitch); act "silu" or "gelu" (its tanh form)."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).gated_act(h, ACTS.get(act))
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_gated_act", got)
    ld, f = _halves(h)
    code = _float_code(h, "h")
    with _on_stream(stream):
        out = torch.empty((h.shape[0], f), dtype=h.dtype, device=h.device)
    _run("gmm_gated_act", _lib().gmm_gated_act(h.data_ptr(), code, h.shape[0], f, ld, _act(act), out.data_ptr(),
                                               _on(h.device, stream)))
    return out


def gated_act_backward(dout, h, act="silu", stream=None):
    """Gradient of gated_act() with respect to h, [rows, 2 f], from dout [rows, f] of h's dtype."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).gated_act_backward(dout, h, ACTS.get(act))
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_gated_act_backward", got)
    ld, f = _halves(h)
    code = _float_code(h, "h")
    _want(dout, "dout", h.dtype, (h.shape[0], f))
    with _on_stream(stream):
        dh = torch.empty((h.shape[0], 2 * f), dtype=h.dtype, device=h.device)
    _run("gmm_gated_act_backward", _lib().gmm_gated_act_backward(
        dout.data_ptr(), h.data_ptr(), code, h.shape[0], f, ld, _act(act), dh.data_ptr(), _on(h.device, stream)))
    return dh


def _group(group, k):
    if group not in INT4_GROUPS:
        raise ValueError(f"group must be one of {INT4_GROUPS}")
    if k < 1 or k % group:
        raise ValueError(f"k must be a multiple of the group ({group}), got {k}")
    return int(group)


def _scales(lead, rows, k, group):
    return lead + (-(-k // _WINDOW), rows, _WINDOW // group)


def quantize_int4(x, group=128, zero_points=False, stream=None):
    """x (bfloat16 or float32) in 4-bit integers with a bfloat16 scale for each `group` values of a
    row, as an Int4Tensor; with zero_points a zero point for each, too, and codes 0 to 15.  x is
    [rows, k] (rows may have a pitch) or a dense [batch, rows, k], the experts' weights for
    matvec_int4()."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).quantize_int4(x, group, 1 if zero_points else 0)
        if got.__class__ is tuple:
            return Int4Tensor(*got, group)
        _run("gmm_quantize_int4", got)
    code = _float_code(x, "x")
    if x.dim() == 3:
        _dev(x, "x")
        batch, rows, k = x.shape
        ld, lead = k, (batch,)
    else:
        ld = _rows(x, "x")
        batch, (rows, k), lead = 1, x.shape, ()
    group = _group(group, k)
    with _on_stream(stream):
        codes = torch.empty(lead + (rows, k // 2), dtype=torch.uint8, device=x.device)
        scale = torch.empty(_scales(lead, rows, k, group), dtype=torch.bfloat16, device=x.device)
        zero = torch.empty(scale.shape, dtype=torch.uint8, device=x.device) if zero_points else None
    _run("gmm_quantize_int4", _lib().gmm_quantize_int4(
        x.data_ptr(), code, batch, rows, k, ld, group, codes.data_ptr(), scale.data_ptr(), _ptr(zero),
        _on(x.device, stream)))
    return Int4Tensor(codes, scale, zero, group)


def _int4_args(q, name):
    """Checks an Int4Tensor; returns its leading dimensions, rows and k."""
    _dev(q.codes, f"{name}.codes")
    if q.codes.dtype != torch.uint8 or q.codes.dim() not in (2, 3):
        raise ValueError(f"{name}.codes must be uint8 [rows, k / 2] or [batch, rows, k / 2]")
    lead, rows, k = tuple(q.codes.shape[:-2]), q.codes.shape[-2], 2 * q.codes.shape[-1]
    shape = _scales(lead, rows, k, _group(q.group, k))
    _want(q.scale, f"{name}.scale", torch.bfloat16, shape)
    if q.zero is not None:
        _want(q.zero, f"{name}.zero", torch.uint8, shape)
    return lead, rows, k


def dequantize_int4(q, out_dtype=torch.bfloat16, stream=None):
    """The values an Int4Tensor stands for, [.., rows, k] of out_dtype (bfloat16 or float32)."""
    if stream is None:
        got = (_moe._calls or _moe._bind()).dequantize_int4(q.codes, q.scale, q.zero, q.group, _OUT_F32.get(out_dtype))
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_dequantize_int4", got)
    lead, rows, k = _int4_args(q, "q")
    with _on_stream(stream):
        out = torch.empty(lead + (rows, k), dtype=out_dtype, device=q.codes.device)
    _run("gmm_dequantize_int4", _lib().gmm_dequantize_int4(
        q.codes.data_ptr(), q.scale.data_ptr(), _ptr(q.zero), q.group, lead[0] if lead else 1, rows, k, out.data_ptr(),
        _float_code(out, "out_dtype"), _on(out.device, stream)))
    return out


def matvec_int4(x, w, experts=None, weights=None, act=None, out_dtype=torch.bfloat16, stream=None):
    """Products of few tokens with the 4-bit weights of the experts that each chose, in the order of
    the tokens: h[t, j] = W[experts[t, j]] x[t], or W[experts[t, j]] x[t, j] for an x of three
    dimensions.  x bfloat16 [tokens, k] (rows may have a pitch of a multiple of 8) or [tokens, topk,
    k]; w an Int4Tensor [E, n, k], n a multiple of 8; experts int32 [tokens, topk].

    Returns h [tokens, topk, n]; with act ("silu" or "gelu") act(first half) * second half, [tokens,
    topk, n / 2] (n a multiple of 16); with weights float32 [tokens, topk] the sum over j of
    weights[t, j] h[t, j], [tokens, n].  Slots outside [0, E) are zeros, and nothing to a sum.
    Without experts w is one matrix [n, k] and h is [tokens, n].  Sums are fp32, rounded once to
    out_dtype (bfloat16 or float32); a row of x with an infinity or NaN gives NaN.

    The matrices are read once for every 8 tokens of an expert (with weights, for every 8 tokens),
    which pays up to some 3 to 8 tokens an expert; past that, sort the rows and use gmm().  It takes
    the codes of groups of 128 without zero points as they are (for up to some 16 rows an expert),
        scale = w.scale.transpose(2, 3).flatten(1, 2)[:, :k // 128, None].float().contiguous()  # once
        gmm(rows, w.codes, sizes, scale, rhs_format="int4")
    and others as dequantize_int4(w)."""
    if stream is None and experts is not None:
        got = (_moe._calls or _moe._bind()).matvec_int4(x, w.codes, w.scale, w.zero, w.group, experts, weights,
                                                        0 if act is None else ACTS.get(act), _OUT_F32.get(out_dtype))
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_matvec_int4", got)
    lead, n, k = _int4_args(w, "w")
    if x.dim() not in (2, 3) or x.shape[-1] != k:
        raise ValueError(f"x must be [tokens, {k}] or [tokens, topk, {k}]")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if experts is None:
        if lead or x.dim() != 2:
            raise ValueError("without experts w must be one matrix and x [tokens, k]")
        topk, num, front = 1, 1, (x.shape[0],)
    else:
        if not lead:
            raise ValueError("with experts w must be [experts, n, k]")
        if experts.dim() != 2 or not 1 <= experts.shape[1] <= MAX_TOPK:
            raise ValueError(f"experts must be [tokens, topk], topk 1..{MAX_TOPK}")
        topk, num, front = experts.shape[1], lead[0], tuple(experts.shape)
        _want(experts, "experts", torch.int32, (x.shape[0], topk))
    if x.dim() == 3:
        _want(x, "x", torch.bfloat16, (x.shape[0], topk, k))
        ld = k
    else:
        ld = _rows(x, "x")
    if weights is not None:
        if experts is None or act is not None:
            raise ValueError("weights go with experts and without act")
        _want(weights, "weights", torch.float32, (x.shape[0], topk))
        front = front[:1]
    code = 0 if act is None else _act(act)
    step = 8 if act is None else 16
    if n < 1 or n % step:
        raise ValueError(f"n must be a multiple of {step}, got {n}")
    if ld % 8:
        raise ValueError("x must have a row pitch that is a multiple of 8")
    lib = _lib()
    nbytes = lib.gmm_matvec_scratch_bytes(x.shape[0], k, w.group, int(w.zero is not None), topk, int(x.dim() == 3))
    with _on_stream(stream):
        scratch = torch.empty((nbytes,), dtype=torch.uint8, device=x.device) if nbytes else None
        out = torch.empty(front + (n if act is None else n // 2,), dtype=out_dtype, device=x.device)
    _run("gmm_matvec_int4", lib.gmm_matvec_int4(
        x.data_ptr(), x.shape[0], k, ld, int(x.dim() == 3), w.codes.data_ptr(), w.scale.data_ptr(), _ptr(w.zero),
        w.group, num, n, _ptr(experts), topk, _ptr(weights), code, out.data_ptr(), _float_code(out, "out_dtype"),
        _ptr(scratch), nbytes, _on(x.device, stream)))
    return out
