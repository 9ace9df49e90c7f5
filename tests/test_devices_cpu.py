"""Tensors of a call have to be on the current device, where the library launches: a kernel given another
device's addresses would fault, or run beside the work that makes its inputs.  The tensors here have a
device and no memory, so nothing could run (no GPU needed)."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B

I32, U8, F32, BF16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def library():
    B.build()
    G.load_library()


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(G, "_current_device", lambda: 0)


def order(z, at):
    return G.ExpertOrder(z("sizes", (4,), I32), z("order.rows", (4, 2), I32), z("order.source", (8,), I32))


def fp4(z, name, *lead, rows=4):
    return G.Fp4Tensor(z(f"{name}.codes", (*lead, rows, 32), U8), z(f"{name}.block_scale", (*lead, 1, rows, 16), U8),
                       z(f"{name}.row_scale", (*lead, rows)), "nvfp4")


CALLS = {
    "route": (lambda z: G.route(z("logits", (4, 8)), 2, select_bias=z("select_bias", (8,)),
                                token_mask=z("token_mask", (4,), torch.bool)), ["logits", "select_bias", "token_mask"]),
    "route_backward": (lambda z: G.route_backward(z("dweights", (4, 2)), z("experts", (4, 2), I32), z("logits", (4, 8))),
                       ["dweights", "experts", "logits"]),
    "sort_by_expert": (lambda z: G.sort_by_expert(z("experts", (4, 2), I32), 4), ["experts"]),
    "dispatch": (lambda z: G.dispatch(z("x", (4, 8)), order(z, 0)), ["x", "order.rows", "order.source"]),
    "combine": (lambda z: G.combine(z("rows", (8, 8)), order(z, 0), z("weights", (4, 2))),
                ["rows", "order.rows", "order.source", "weights"]),
    "combine_backward": (lambda z: G.combine_backward(z("dout", (4, 8)), z("rows", (8, 8)), order(z, 0), z("weights", (4, 2))),
                         ["dout", "rows", "order.rows", "order.source", "weights"]),
    "quantize_fp4": (lambda z: G.quantize_fp4(z("x", (4, 64)), order=order(z, 0)), ["x", "order.rows", "order.source"]),
    "quantize_fp4 batch": (lambda z: G.quantize_fp4(z("x", (2, 4, 64))), ["x"]),
    "dequantize_fp4": (lambda z: G.dequantize_fp4(fp4(z, "q")), ["q.codes", "q.block_scale", "q.row_scale"]),
    "gmm_fp4": (lambda z: G.gmm_fp4(fp4(z, "lhs"), fp4(z, "rhs", 2, rows=8), z("group_sizes", (2,), I32),
                                    workspace=z("workspace", (256,), U8)),
                ["lhs.codes", "lhs.block_scale", "lhs.row_scale", "rhs.codes", "rhs.block_scale", "rhs.row_scale",
                 "group_sizes", "workspace"]),
    "gmm": (lambda z: G.gmm(z("lhs", (4, 8), BF16), z("rhs", (2, 8, 8), BF16), z("group_sizes", (2,), I32),
                            workspace=z("workspace", (256,), U8), out=z("out", (4, 8), BF16)),
            ["lhs", "rhs", "group_sizes", "out"]),
    "tgmm": (lambda z: G.tgmm(z("lhs", (4, 8), BF16), z("dout", (4, 8), BF16), z("group_sizes", (2,), I32),
                              workspace=z("workspace", (256,), U8), out=z("out", (2, 8, 8))),
             ["lhs", "dout", "group_sizes", "out"]),
}


@pytest.mark.parametrize("name,operand", [(n, o) for n, (_, operands) in CALLS.items() for o in [*operands, "all"]])
def test_a_tensor_of_another_device_is_refused(current, name, operand):
    with FakeTensorMode():
        def z(what, shape, dtype=F32):
            return torch.empty(shape, dtype=dtype, device="cuda:1" if operand in (what, "all") else "cuda:0")

        with pytest.raises(ValueError, match="is on cuda:1, but the current device is cuda:0") as e:
            CALLS[name][0](z)
    assert operand == "all" or str(e.value).startswith(operand + " ")
