"""The operators around the grouped products of a mixture-of-experts layer, behind the C ABI of
libgmm (``include/libgmm_moe.h``): the router's choice of experts, the tokens' rows sorted by
expert and brought back, and microscaled 4-bit floating point.

    weights, experts = route(logits, topk)
    order = sort_by_expert(experts, num_experts)
    rows = dispatch(x, order)                      # the experts' input rows, for gmm()
    out = combine(rows_out, order, weights)        # back in token order
    q = quantize_fp4(x, "nvfp4", order=order)      # the same rows in 4 bits, for gmm_fp4()

Like the rest of the package this only marshals arguments; gradients are calls of their own
(``route_backward``, ``dispatch_backward``, ``combine_backward``).  A call with ``stream=`` runs on
that stream and its results belong to it, as if it were made under ``torch.cuda.stream(stream)``;
its inputs are the caller's to keep ready and alive for it.  Arguments that are right as they
stand go to the library through ``csrc/host_calls.cpp`` in one step; all others
are looked at here, one by one, and called through ctypes or refused.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import sys
import warnings
from typing import NamedTuple, Optional

import torch

from . import (_I, _I32, _I64, _P, _SZ, DTYPE_BF16, DTYPE_F32, SIGNATURES, GmmError, _dev, _here, _on_stream,
               load_library, workspace_for)

__all__ = ["route", "route_backward", "ExpertOrder", "sort_by_expert", "dispatch", "dispatch_backward", "combine",
           "combine_backward", "Fp4Tensor", "quantize_fp4", "dequantize_fp4", "gmm_fp4", "MAX_TOPK"]

SCORES = {"softmax": 0, "sigmoid": 1}
_BIASED = {"softmax": 16, "sigmoid": 17}
FP4_FORMATS = {"nvfp4": 0, "mxfp4": 1}
FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}
MAX_TOPK = 32
_OUT_F32 = {torch.bfloat16: 0, torch.float32: 1}

_package = sys.modules[__package__]
_F = ctypes.c_float
SIGNATURES.update({
    "gmm_route": ([_P, _I, _I64, _I32, _I64, _I32, _I, _I, _F, _P, _P, _P, _P, _P], _I),
    "gmm_route_backward": ([_P, _P, _P, _I, _I64, _I32, _I64, _I32, _I, _I, _F, _P, _P], _I),
    "gmm_sort_by_expert": ([_P, _I64, _I32, _I32, _P, _P, _P, _P], _I),
    "gmm_dispatch": ([_P, _I, _I64, _I64, _I64, _I32, _P, _P, _P, _P], _I),
    "gmm_combine": ([_P, _I, _I64, _I64, _I32, _P, _P, _P, _P], _I),
    "gmm_combine_backward": ([_P, _P, _I, _I64, _I64, _I32, _P, _P, _P, _P, _P, _P], _I),
    "gmm_quantize_fp4": ([_P, _I, _I32, _I64, _I64, _I64, _I, _P, _P, _I32, _P, _P, _P, _P], _I),
    "gmm_dequantize_fp4": ([_P, _P, _P, _I, _I32, _I64, _I64, _P, _I, _P], _I),
    "gmm_fp4": ([_P, _P, _P, _I64, _I64, _P, _P, _P, _I, _I32, _I64, _P, _I32, _I32, _P, _I, _P, _I, _P, _SZ, _P], _I),
})


class ExpertOrder(NamedTuple):
    """The slots of a [tokens, topk] choice sorted by expert: int32 tensors group_sizes [experts],
    rows [tokens, topk] (the row of each slot, -1 if dropped) and source [tokens * topk] (the slot
    of each row, -1 past the groups)."""
    group_sizes: torch.Tensor
    rows: torch.Tensor
    source: torch.Tensor


class Fp4Tensor(NamedTuple):
    """Matrices [.., rows, k] of e2m1 codes: codes uint8 [.., rows, k / 2] (even k in the low
    nibble), block_scale uint8 [.., windows, rows, 16] (16 blocks a window; e4m3 bytes a block of
    16 for "nvfp4", E8M0 bytes a block of 32 for "mxfp4"; bytes past the last block are 0: gmm_fp4()
    reads whole windows, and a NaN there would reach its sums), row_scale float32 [.., rows]
    ("nvfp4") or None."""
    codes: torch.Tensor
    block_scale: torch.Tensor
    row_scale: Optional[torch.Tensor]
    format: str


# These calls are a few microseconds of GPU work at decoding sizes, so the checks below cost as
# little as they can: one test that holds for good arguments, and the reason only where it fails.
# A PyTorch without CUDA has no such function, and no tensor that any call takes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(device, stream):
    """The CUDA stream handle of `stream`, or of the device's current stream."""
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _run(fn, status):
    """Raises for a status that is not 0 (None: there is none)."""
    if status:
        raise GmmError(fn, status)


def _lib():
    return _package._lib or load_library()


_calls = None


class _NoCalls:
    """Stands for host-side calls that are not there: none takes any arguments."""

    def __getattr__(self, name):
        return lambda *args: None


def _bind():
    """Loads the host-side calls built for this PyTorch and gives them the loaded library's functions;
    without them every call goes through the checks below and ctypes."""
    global _calls
    from .build import host_calls_path

    lib = load_library()
    path = host_calls_path()
    loader = importlib.machinery.ExtensionFileLoader(f"{__package__}._host_calls", path)
    try:
        calls = importlib.util.module_from_spec(importlib.util.spec_from_file_location(loader.name, path, loader=loader))
        loader.exec_module(calls)
        names = ("gmm_route", "gmm_route_backward", "gmm_sort_by_expert", "gmm_dispatch", "gmm_combine",
                 "gmm_combine_backward", "gmm_quantize_fp4", "gmm_dequantize_fp4", "gmm_fp4",
                 "gmm_balance_scratch_bytes", "gmm_balance_loss", "gmm_balance_loss_backward", "gmm_gated_act",
                 "gmm_gated_act_backward", "gmm_quantize_int4", "gmm_dequantize_int4", "gmm_matvec_int4",
                 "gmm_matvec_scratch_bytes")
        calls.bind(*[ctypes.cast(getattr(lib, n), _P).value for n in names])
    except ImportError as e:
        warnings.warn(f"the mixture-of-experts calls go the longer way, some 7 us of host time more for each ({e}): "
                      "build with `python -m moe_grouped_matrix_gb300.build`", RuntimeWarning, stacklevel=3)
        calls = _NoCalls()
    _calls = calls
    return calls


def _rows(t, name):
    """A 2-D CUDA tensor whose rows are dense; returns its row pitch."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _here(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    n, d = t.shape
    pitch, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{name} must have dense rows")
    if n <= 1:
        return d
    if pitch < d:
        raise ValueError(f"{name} must have rows that do not overlap")
    return pitch


_FLOATS = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}


def _float_code(t, name):
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32")
    return code


def _want(t, name, dtype, shape):
    _dev(t, name)
    if t.dtype is dtype and t.shape == shape:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _biased(bias_on):
    """The scores' codes where select_bias is not the logit's."""
    if bias_on != "score":
        raise ValueError("bias_on must be 'logit' or 'score'")
    return _BIASED


def _score(score, codes=SCORES):
    try:
        return codes[score]
    except KeyError:
        raise ValueError(f"score must be one of {sorted(SCORES)}") from None


def route(logits, topk, score="softmax", renormalize=True, scale=1.0, select_bias=None, token_mask=None, stream=None,
          bias_on="logit"):
    """The topk experts of each token and their weights: (weights float32 [tokens, topk], experts
    int32 [tokens, topk]) from logits [tokens, experts] (bfloat16 or float32, rows may have a
    pitch).  Experts are chosen by logit + select_bias (float32 [experts]), largest first, equal
    ones by index; experts whose logit is -inf or NaN are never chosen.  With bias_on="score" they
    are chosen by softmax (over all experts) or sigmoid + select_bias, the form of biases that
    balance the experts' loads: the two choose different experts.  The bias moves the choice only,
    never the weights.  Weights are
    scale * softmax (over all experts) or scale * sigmoid of the logits, divided by their sum over
    the chosen experts with renormalize.  Tokens whose token_mask (bool or uint8 [tokens]) is 0,
    and slots past the experts that can be chosen, have expert -1 and weight 0."""
    if stream is None:
        got = (_calls or _bind()).route(logits, topk, (SCORES if bias_on == "logit" else _biased(bias_on)).get(score),
                                        1 if renormalize else 0, scale, select_bias, token_mask)
        if got.__class__ is tuple:
            return got
        _run("gmm_route", got)
    ld = _rows(logits, "logits")
    code = _float_code(logits, "logits")
    tokens, experts = logits.shape
    topk = int(topk)
    if not 1 <= topk <= min(experts, MAX_TOPK):
        raise ValueError(f"topk must be 1..{min(experts, MAX_TOPK)}")
    if select_bias is not None:
        _want(select_bias, "select_bias", torch.float32, (experts,))
    if token_mask is not None:
        _want(token_mask, "token_mask", torch.uint8 if token_mask.dtype == torch.uint8 else torch.bool, (tokens,))
    with _on_stream(stream):
        weights = torch.empty((tokens, topk), dtype=torch.float32, device=logits.device)
        chosen = torch.empty((tokens, topk), dtype=torch.int32, device=logits.device)
    _run("gmm_route", _lib().gmm_route(
        logits.data_ptr(), code, tokens, experts, ld, topk,
        _score(score, SCORES if bias_on == "logit" else _biased(bias_on)), int(bool(renormalize)), float(scale),
        _ptr(select_bias), _ptr(token_mask), weights.data_ptr(), chosen.data_ptr(), _on(logits.device, stream)))
    return weights, chosen


def route_backward(dweights, experts, logits, score="softmax", renormalize=True, scale=1.0, stream=None):
    """Gradient of route()'s weights with respect to the logits, [tokens, experts] of the logits'
    dtype, from dweights float32 [tokens, topk] and the experts that route() chose."""
    if stream is None:
        got = (_calls or _bind()).route_backward(dweights, experts, logits, SCORES.get(score),
                                                 1 if renormalize else 0, scale)
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_route_backward", got)
    ld = _rows(logits, "logits")
    code = _float_code(logits, "logits")
    tokens, n = logits.shape
    if experts.dim() != 2:
        raise ValueError("experts must be [tokens, topk]")
    topk = experts.shape[1]
    _want(experts, "experts", torch.int32, (tokens, topk))
    _want(dweights, "dweights", torch.float32, (tokens, topk))
    with _on_stream(stream):
        dlogits = torch.empty((tokens, n), dtype=logits.dtype, device=logits.device)
    _run("gmm_route_backward", _lib().gmm_route_backward(
        dweights.data_ptr(), experts.data_ptr(), logits.data_ptr(), code, tokens, n, ld, topk, _score(score),
        int(bool(renormalize)), float(scale), dlogits.data_ptr(), _on(logits.device, stream)))
    return dlogits


def sort_by_expert(experts, num_experts, stream=None):
    """The stable order of the slots of experts int32 [tokens, topk] by expert, as an ExpertOrder.
    Slots whose expert is outside [0, num_experts) are dropped."""
    if stream is None:
        got = (_calls or _bind()).sort_by_expert(experts, num_experts)
        if got.__class__ is tuple:
            return ExpertOrder._make(got)
        _run("gmm_sort_by_expert", got)
    if experts.dim() != 2:
        raise ValueError("experts must be [tokens, topk]")
    tokens, topk = experts.shape
    _want(experts, "experts", torch.int32, (tokens, topk))
    with _on_stream(stream):
        sizes = torch.empty((int(num_experts),), dtype=torch.int32, device=experts.device)
        rows = torch.empty((tokens, topk), dtype=torch.int32, device=experts.device)
        source = torch.empty((tokens * topk,), dtype=torch.int32, device=experts.device)
    _run("gmm_sort_by_expert", _lib().gmm_sort_by_expert(
        experts.data_ptr(), tokens, topk, int(num_experts), sizes.data_ptr(), rows.data_ptr(), source.data_ptr(),
        _on(experts.device, stream)))
    return ExpertOrder(sizes, rows, source)


def _order(order):
    if order.rows.dim() != 2:
        raise ValueError("order.rows must be [tokens, topk]")
    tokens, topk = order.rows.shape
    _want(order.rows, "order.rows", torch.int32, (tokens, topk))
    _want(order.source, "order.source", torch.int32, (tokens * topk,))
    return tokens, topk


def dispatch(x, order, stream=None):
    """The rows of x [tokens, d] (bfloat16 or float32, rows may have a pitch) in expert order:
    [tokens * topk, d], zeros past the groups."""
    if stream is None:
        got = (_calls or _bind()).dispatch(x, order.rows, order.source)
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_dispatch", got)
    ld = _rows(x, "x")
    code = _float_code(x, "x")
    tokens, topk = _order(order)
    if x.shape[0] != tokens:
        raise ValueError(f"x must have {tokens} rows")
    with _on_stream(stream):
        out = torch.empty((tokens * topk, x.shape[1]), dtype=x.dtype, device=x.device)
    _run("gmm_dispatch", _lib().gmm_dispatch(
        x.data_ptr(), code, tokens, x.shape[1], ld, topk, order.rows.data_ptr(), order.source.data_ptr(),
        out.data_ptr(), _on(x.device, stream)))
    return out


def combine(rows, order, weights=None, stream=None):
    """Token order again: out[t] = sum over t's slots of weights[t, j] * rows[order.rows[t, j]], in
    fp32, rounded once; weights float32 [tokens, topk], or None for ones.  rows [tokens * topk, d]."""
    if stream is None:
        got = (_calls or _bind()).combine(rows, order.rows, order.source, weights)
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_combine", got)
    code = _float_code(_dev(rows, "rows"), "rows")
    tokens, topk = _order(order)
    if rows.dim() != 2 or rows.shape[0] != tokens * topk:
        raise ValueError(f"rows must be [{tokens * topk}, d]")
    if weights is not None:
        _want(weights, "weights", torch.float32, (tokens, topk))
    with _on_stream(stream):
        out = torch.empty((tokens, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    _run("gmm_combine", _lib().gmm_combine(
        rows.data_ptr(), code, tokens, rows.shape[1], topk, order.rows.data_ptr(), _ptr(weights), out.data_ptr(),
        _on(rows.device, stream)))
    return out


def dispatch_backward(drows, order, stream=None):
    """Gradient of dispatch() with respect to x: the sum of each token's rows of drows."""
    return combine(drows, order, None, stream)


def combine_backward(dout, rows, order, weights, stream=None):
    """Gradients of combine(): (drows [tokens * topk, d] of the rows' dtype, dweights float32
    [tokens, topk]) from dout [tokens, d] of the rows' dtype."""
    if stream is None:
        got = (_calls or _bind()).combine_backward(dout, rows, order.rows, order.source, weights)
        if got.__class__ is tuple:
            return got
        _run("gmm_combine_backward", got)
    code = _float_code(_dev(rows, "rows"), "rows")
    tokens, topk = _order(order)
    if rows.dim() != 2 or rows.shape[0] != tokens * topk:
        raise ValueError(f"rows must be [{tokens * topk}, d]")
    _want(dout, "dout", rows.dtype, (tokens, rows.shape[1]))
    _want(weights, "weights", torch.float32, (tokens, topk))
    with _on_stream(stream):
        drows = torch.empty_like(rows)
        dweights = torch.empty((tokens, topk), dtype=torch.float32, device=rows.device)
    _run("gmm_combine_backward", _lib().gmm_combine_backward(
        dout.data_ptr(), rows.data_ptr(), code, tokens, rows.shape[1], topk, order.rows.data_ptr(),
        order.source.data_ptr(), weights.data_ptr(), drows.data_ptr(), dweights.data_ptr(),
        _on(rows.device, stream)))
    return drows, dweights


def _fp4_format(fmt):
    try:
        return FP4_FORMATS[fmt]
    except KeyError:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}") from None


def _windows(k, fmt):
    return -(-k // (16 * FP4_BLOCK[fmt]))


def quantize_fp4(x, format="nvfp4", order=None, stream=None):
    """x (bfloat16 or float32) in microscaled 4-bit floating point, as an Fp4Tensor.  x is
    [rows, k] (rows may have a pitch) or a dense [batch, rows, k], the experts' weights for
    gmm_fp4(); k must be a multiple of 32.  With order, x [tokens, k] gives the rows of
    dispatch(x, order), each token quantised once."""
    if stream is None:
        got = (_calls or _bind()).quantize_fp4(x, FP4_FORMATS.get(format), None if order is None else order.rows,
                                               None if order is None else order.source)
        if got.__class__ is tuple:
            return Fp4Tensor(*got, format)
        _run("gmm_quantize_fp4", got)
    fmt = _fp4_format(format)
    code = _float_code(x, "x")
    if x.dim() == 3:
        _dev(x, "x")
        batch, rows, k = x.shape
        ld, lead = k, (batch,)
    else:
        ld = _rows(x, "x")
        batch, (rows, k), lead = 1, x.shape, ()
    topk, out_rows = 1, rows
    if order is not None:
        tokens, topk = _order(order)
        if x.dim() != 2 or rows != tokens:
            raise ValueError(f"with an order x must be [{tokens}, k]")
        out_rows = tokens * topk
    if k % 32:
        raise ValueError("k must be a multiple of 32")
    with _on_stream(stream):
        codes = torch.empty(lead + (out_rows, k // 2), dtype=torch.uint8, device=x.device)
        scale = torch.empty(lead + (_windows(k, format), out_rows, 16), dtype=torch.uint8, device=x.device)
        row = torch.empty(lead + (out_rows,), dtype=torch.float32, device=x.device) if format == "nvfp4" else None
    if batch == 0:
        return Fp4Tensor(codes, scale, row, format)
    _run("gmm_quantize_fp4", _lib().gmm_quantize_fp4(
        x.data_ptr(), code, batch, rows, k, ld, fmt, None if order is None else order.rows.data_ptr(),
        None if order is None else order.source.data_ptr(), topk, codes.data_ptr(), scale.data_ptr(), _ptr(row),
        _on(x.device, stream)))
    return Fp4Tensor(codes, scale, row, format)


def _fp4_args(q, name, lead):
    """Checks an Fp4Tensor with `lead` leading dimensions; returns (rows, k)."""
    fmt = q.format
    _fp4_format(fmt)
    _dev(q.codes, f"{name}.codes")
    if q.codes.dtype != torch.uint8 or q.codes.dim() != lead + 2:
        raise ValueError(f"{name}.codes must be uint8 with {lead + 2} dimensions")
    front, rows, k = tuple(q.codes.shape[:lead]), q.codes.shape[-2], 2 * q.codes.shape[-1]
    _want(q.block_scale, f"{name}.block_scale", torch.uint8, front + (_windows(k, fmt), rows, 16))
    if fmt == "nvfp4":
        if q.row_scale is None:
            raise ValueError(f"{name}.row_scale is needed for nvfp4")
        _want(q.row_scale, f"{name}.row_scale", torch.float32, front + (rows,))
    elif q.row_scale is not None:
        raise ValueError(f"{name}.row_scale must be None for mxfp4")
    return rows, k


def dequantize_fp4(q, out_dtype=torch.bfloat16, stream=None):
    """The values an Fp4Tensor stands for, [.., rows, k] of out_dtype (bfloat16 or float32)."""
    if stream is None:
        got = (_calls or _bind()).dequantize_fp4(q.codes, q.block_scale, q.row_scale, FP4_FORMATS.get(q.format),
                                                 _OUT_F32.get(out_dtype))
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_dequantize_fp4", got)
    lead = q.codes.dim() - 2
    if lead not in (0, 1):
        raise ValueError("codes must be [rows, k / 2] or [batch, rows, k / 2]")
    rows, k = _fp4_args(q, "q", lead)
    batch = q.codes.shape[0] if lead else 1
    with _on_stream(stream):
        out = torch.empty(tuple(q.codes.shape[:-1]) + (k,), dtype=out_dtype, device=q.codes.device)
    if batch == 0:
        return out
    _run("gmm_dequantize_fp4", _lib().gmm_dequantize_fp4(
        q.codes.data_ptr(), q.block_scale.data_ptr(), _ptr(q.row_scale), FP4_FORMATS[q.format], batch, rows, k,
        out.data_ptr(), _float_code(out, "out_dtype"), _on(out.device, stream)))
    return out


def gmm_fp4(lhs, rhs, group_sizes, rhs_bias=None, group_offset=0, out=None, out_dtype=torch.bfloat16, workspace=None,
            stream=None):
    """out[r] = lhs[r] @ W_g^T for each row r of local group g, all other rows zero, as gmm() with the
    NT layout: lhs an Fp4Tensor [m, k], rhs an Fp4Tensor [G_local, n, k] of the same format, on the
    block-scaled 4-bit tensor cores.  k must be a multiple of 32 and n of 8; rhs_bias
    [G_local, 1, n] bfloat16 or float32; group_offset an int (gmm()'s may be on the device)."""
    if stream is None and rhs_bias is None and out is None and lhs.format == rhs.format and lhs.codes.is_cuda:
        ws = workspace
        if ws is None:
            index = lhs.codes.device.index
            ws = _package._workspaces.get((index, _raw_stream(index)))  # workspace_for()'s
        got = (_calls or _bind()).gmm_fp4(lhs.codes, lhs.block_scale, lhs.row_scale, rhs.codes, rhs.block_scale,
                                          rhs.row_scale, FP4_FORMATS.get(lhs.format), group_sizes, group_offset,
                                          _OUT_F32.get(out_dtype), ws)
        if got.__class__ is torch.Tensor:
            return got
        _run("gmm_fp4", got)
    m, k = _fp4_args(lhs, "lhs", 0)
    n, kr = _fp4_args(rhs, "rhs", 1)
    if kr != k:
        raise ValueError(f"lhs has k={k} but rhs has k={kr}")
    if lhs.format != rhs.format:
        raise ValueError(f"lhs is {lhs.format} but rhs is {rhs.format}")
    local = rhs.codes.shape[0]
    _dev(group_sizes, "group_sizes")
    if group_sizes.dtype != torch.int32:
        raise TypeError("group_sizes must be int32")
    device = lhs.codes.device
    if rhs_bias is not None:
        _want(rhs_bias, "rhs_bias", rhs_bias.dtype, (local, 1, n))
        bias_code = _float_code(rhs_bias, "rhs_bias")
    else:
        bias_code = DTYPE_BF16
    if out is None:
        with _on_stream(stream):
            out = torch.empty((m, n), dtype=out_dtype, device=device)
    _dev(out, "out")
    if tuple(out.shape) != (m, n):
        raise ValueError(f"out must be [{m}, {n}], got {list(out.shape)}")
    ws = workspace if workspace is not None else workspace_for(device, stream)
    _dev(ws, "workspace")
    _run("gmm_fp4", _lib().gmm_fp4(
        lhs.codes.data_ptr(), lhs.block_scale.data_ptr(), _ptr(lhs.row_scale), m, k, rhs.codes.data_ptr(),
        rhs.block_scale.data_ptr(), _ptr(rhs.row_scale), FP4_FORMATS[lhs.format], local, n, group_sizes.data_ptr(),
        group_sizes.shape[0], int(group_offset), _ptr(rhs_bias), bias_code, out.data_ptr(),
        _float_code(out, "out"), ws.data_ptr(), ws.numel(), _on(device, stream)))
    return out
