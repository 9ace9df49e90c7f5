"""The binding's short way (csrc/host_calls.cpp) and its longer one (moe.py) take the same arguments, refuse
the same, and give the same bits."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import moe
from test_moe_streams_gpu import CALLS, DEV, data, same  # noqa: F401

pytestmark = pytest.mark.gpu


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def i(*shape):
    return t(*shape, dtype=torch.int32)


def fp4(fmt, *lead, rows=4, k=64, **over):
    windows = -(-k // (256 if fmt == "nvfp4" else 512))
    parts = dict(codes=t(*lead, rows, k // 2, dtype=torch.uint8), block_scale=t(*lead, windows, rows, 16, dtype=torch.uint8),
                 row_scale=t(*lead, rows) if fmt == "nvfp4" else None, format=fmt)
    return G.Fp4Tensor(**{**parts, **over})


def order(tokens=4, topk=2, **over):
    parts = dict(group_sizes=i(4), rows=i(tokens, topk), source=i(tokens * topk))
    return G.ExpertOrder(**{**parts, **over})


class Odd(torch.Tensor):
    pass


ARGUMENTS = {
    "route float topk": lambda: G.route(t(4, 8), 2.0),
    "route bool topk": lambda: G.route(t(4, 8), True),
    "route topk 0": lambda: G.route(t(4, 8), 0),
    "route topk 9": lambda: G.route(t(4, 8), 9),
    "route topk 33": lambda: G.route(t(4, 64), 33),
    "route huge topk": lambda: G.route(t(4, 8), 2 ** 70),
    "route no experts": lambda: G.route(t(4, 0), 1),
    "route 1025": lambda: G.route(t(4, 1025), 2),
    "route 1-d": lambda: G.route(t(8), 2),
    "route half": lambda: G.route(t(4, 8).half(), 2),
    "route columns": lambda: G.route(t(8, 4).t(), 2),
    "route every other column": lambda: G.route(t(4, 16)[:, ::2], 2),
    "route one column": lambda: G.route(t(4, 8)[:, :1], 1),
    "route expanded": lambda: G.route(t(1, 8).expand(4, 8), 2),
    "route one expanded row": lambda: G.route(t(1, 8).expand(1, 8), 2),
    "route score": lambda: G.route(t(4, 8), 2, "tanh"),
    "route bias length": lambda: G.route(t(4, 8), 2, select_bias=t(7)),
    "route bias type": lambda: G.route(t(4, 8), 2, select_bias=t(8).half()),
    "route bias strided": lambda: G.route(t(4, 8), 2, select_bias=t(16)[::2]),
    "route mask type": lambda: G.route(t(4, 8), 2, token_mask=t(4)),
    "route mask length": lambda: G.route(t(4, 8), 2, token_mask=t(5, dtype=torch.bool)),
    "route host": lambda: G.route(torch.zeros(4, 8), 2),
    "route subclass": lambda: G.route(t(4, 8).as_subclass(Odd), 2),
    "route parameter": lambda: G.route(torch.nn.Parameter(t(4, 8)), 2),
    "route_backward types": lambda: G.route_backward(t(4, 2), t(4, 2), t(4, 8)),
    "route_backward shapes": lambda: G.route_backward(t(4, 3), i(4, 2), t(4, 8)),
    "route_backward topk": lambda: G.route_backward(t(4, 9), i(4, 9), t(4, 8)),
    "route_backward tokens": lambda: G.route_backward(t(3, 2), i(3, 2), t(4, 8)),
    "sort 1-d": lambda: G.sort_by_expert(i(8), 4),
    "sort long": lambda: G.sort_by_expert(i(4, 2).long(), 4),
    "sort none": lambda: G.sort_by_expert(i(4, 2), 0),
    "sort 1025": lambda: G.sort_by_expert(i(4, 2), 1025),
    "sort topk 33": lambda: G.sort_by_expert(i(4, 33), 4),
    "sort strided": lambda: G.sort_by_expert(i(4, 4)[:, :2], 4),
    "dispatch tokens": lambda: G.dispatch(t(3, 8), order()),
    "dispatch source": lambda: G.dispatch(t(4, 8), order(source=i(7))),
    "dispatch rows": lambda: G.dispatch(t(4, 8), order(rows=i(8))),
    "dispatch half": lambda: G.dispatch(t(4, 8).half(), order()),
    "dispatch no columns": lambda: G.dispatch(t(4, 0), order()),
    "dispatch overlapping": lambda: G.dispatch(t(16).as_strided((4, 8), (2, 1)), order()),
    "combine rows": lambda: G.combine(t(7, 8), order()),
    "combine strided": lambda: G.combine(t(8, 16)[:, :8], order()),
    "combine weights": lambda: G.combine(t(8, 8), order(), t(4, 3)),
    "combine weights half": lambda: G.combine(t(8, 8), order(), t(4, 2).half()),
    "combine_backward types": lambda: G.combine_backward(t(4, 8).bfloat16(), t(8, 8), order(), t(4, 2)),
    "combine_backward shapes": lambda: G.combine_backward(t(4, 9), t(8, 8), order(), t(4, 2)),
    "combine_backward weights": lambda: G.combine_backward(t(4, 8), t(8, 8), order(), t(8)),
    "quantize k": lambda: G.quantize_fp4(t(4, 48)),
    "quantize k 0": lambda: G.quantize_fp4(t(4, 0)),
    "quantize format": lambda: G.quantize_fp4(t(4, 64), "fp5"),
    "quantize 1-d": lambda: G.quantize_fp4(t(64)),
    "quantize tokens": lambda: G.quantize_fp4(t(3, 64), order=order()),
    "quantize expanded": lambda: G.quantize_fp4(t(1, 64).expand(4, 64)),
    "dequantize scale": lambda: G.dequantize_fp4(fp4("nvfp4", block_scale=t(1, 5, 16, dtype=torch.uint8))),
    "dequantize no row scale": lambda: G.dequantize_fp4(fp4("nvfp4", row_scale=None)),
    "dequantize row scale": lambda: G.dequantize_fp4(fp4("mxfp4", row_scale=t(4))),
    "dequantize format": lambda: G.dequantize_fp4(fp4("nvfp4", format="fp5")),
    "dequantize out": lambda: G.dequantize_fp4(fp4("nvfp4"), torch.float16),
    "product formats": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("mxfp4", 2, rows=8), i(2)),
    "product depth": lambda: G.gmm_fp4(fp4("nvfp4", k=96), fp4("nvfp4", 2, rows=8), i(2)),
    "product columns": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=12), i(2)),
    "product groups": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(1)),
    "product sizes long": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(2).long()),
    "product offset": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(3), group_offset=2),
    "product negative offset": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(3), group_offset=-1),
    "product out type": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(2), out_dtype=torch.float16),
    "product 2-d weights": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", rows=8), i(2)),
    "product workspace": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(2), workspace=t(64, dtype=torch.uint8)),
    "product slice": lambda: G.gmm_fp4(fp4("nvfp4"), fp4("nvfp4", 2, rows=8), i(3), group_offset=1),
}


def outcome(call):
    try:
        return call(), None
    except (TypeError, ValueError, RuntimeError) as e:
        return None, (type(e), str(e))


@pytest.mark.parametrize("name", sorted(CALLS) + sorted(ARGUMENTS))
def test_both_ways_agree(data, name, monkeypatch):  # noqa: F811
    call = ARGUMENTS[name] if name in ARGUMENTS else lambda: CALLS[name](data)
    short = outcome(call)
    assert not isinstance(moe._calls or moe._bind(), moe._NoCalls)
    monkeypatch.setattr(moe, "_calls", moe._NoCalls())
    long = outcome(call)
    torch.cuda.synchronize()
    assert short[1] == long[1]
    assert short[1] is not None or same(short[0], long[0])
