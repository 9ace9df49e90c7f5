"""The operators of include/libgmm_experts.h: exported, bound, and refusing bad host-side arguments
before anything touches a device (no GPU needed)."""

import ctypes
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "libgmm_experts.h")
P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)
ODD8 = ctypes.c_void_p((1 << 20) + 8)
NULL, DTYPE, SHAPE, ALIGN, WORKSPACE, ARCH, CUDA = 1, 2, 3, 4, 6, 7, 8
LARGEST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load_library()


def test_every_declared_call_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^(?:int|size_t)\s+(gmm_[a-z0-9_]+)\s*\(", text, flags=re.M)
    assert len(names) == 9
    for name in names:
        assert hasattr(lib, name) and name in G.SIGNATURES
        args = re.search(re.escape(name) + r"\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(args.split(",")) == len(G.SIGNATURES[name][0]), name


LOSS = dict(logits=P, dtype=1, tokens=8, experts=8, ld=8, chosen=P, topk=2, score=0, mask=None, sequences=2, losses=P,
            counts=P, counted=P, scratch=P, scratch_bytes=1 << 20, stream=None)
LBACK = dict(dlosses=P, counts=P, counted=P, logits=P, dtype=1, tokens=8, experts=8, ld=8, score=0, mask=None,
             sequences=2, dlogits=P, stream=None)
ACT = dict(h=P, dtype=0, rows=4, f=8, ld=16, act=1, out=P, stream=None)
ABACK = dict(dout=P, h=P, dtype=0, rows=4, f=8, ld=16, act=1, dh=P, stream=None)
QUANT = dict(x=P, dtype=0, batch=1, rows=4, k=256, ld=256, group=64, codes=P, scale=P, zero=P, stream=None)
DEQUANT = dict(codes=P, scale=P, zero=P, group=64, batch=1, rows=4, k=256, out=P, dtype=0, stream=None)
VEC = dict(x=P, tokens=4, k=256, ld=256, per_slot=0, codes=P, scale=P, zero=None, group=64, experts=8, n=32, chosen=P,
           topk=2, weights=None, act=0, out=P, out_dtype=0, scratch=None, scratch_bytes=0, stream=None)

REFUSALS = [
    ("gmm_balance_loss", LOSS, NULL, [dict(logits=None), dict(chosen=None), dict(losses=None), dict(counts=None),
                                      dict(counted=None), dict(tokens=0, losses=None)]),
    ("gmm_balance_loss", LOSS, DTYPE, [dict(dtype=2)]),
    ("gmm_balance_loss", LOSS, SHAPE, [dict(tokens=-2), dict(tokens=9), dict(sequences=0), dict(sequences=3),
                                       dict(experts=0), dict(experts=1025, ld=1025), dict(ld=7), dict(topk=0),
                                       dict(topk=33), dict(score=2), dict(score=16),
                                       dict(tokens=LARGEST, topk=2), dict(tokens=LARGEST + 2, topk=1)]),
    ("gmm_balance_loss", LOSS, ALIGN, [dict(logits=ODD), dict(chosen=ODD), dict(losses=ODD), dict(counts=ODD),
                                       dict(counted=ODD), dict(scratch=ODD8)]),
    ("gmm_balance_loss", LOSS, WORKSPACE, [dict(scratch_bytes=0), dict(scratch_bytes=100), dict(scratch=None)]),
    ("gmm_balance_loss_backward", LBACK, NULL, [dict(dlosses=None), dict(counts=None), dict(counted=None),
                                                dict(logits=None), dict(dlogits=None)]),
    ("gmm_balance_loss_backward", LBACK, DTYPE, [dict(dtype=3)]),
    ("gmm_balance_loss_backward", LBACK, SHAPE, [dict(sequences=3), dict(ld=7), dict(score=2)]),
    ("gmm_balance_loss_backward", LBACK, ALIGN, [dict(dlogits=ODD), dict(dlosses=ODD)]),
    ("gmm_gated_act", ACT, NULL, [dict(h=None), dict(out=None)]),
    ("gmm_gated_act", ACT, DTYPE, [dict(dtype=2)]),
    ("gmm_gated_act", ACT, SHAPE, [dict(rows=-1), dict(f=0), dict(ld=15), dict(act=0), dict(act=3),
                                   dict(f=2 ** 28, ld=2 ** 30), dict(rows=LARGEST + 1)]),
    ("gmm_gated_act", ACT, ALIGN, [dict(dtype=1, h=ODD), dict(dtype=1, out=ODD), dict(h=ctypes.c_void_p(4097))]),
    ("gmm_gated_act_backward", ABACK, NULL, [dict(dout=None), dict(h=None), dict(dh=None)]),
    ("gmm_gated_act_backward", ABACK, SHAPE, [dict(ld=15), dict(act=0)]),
    ("gmm_gated_act_backward", ABACK, ALIGN, [dict(dtype=1, dout=ODD)]),
    ("gmm_quantize_int4", QUANT, NULL, [dict(x=None), dict(codes=None), dict(scale=None)]),
    ("gmm_quantize_int4", QUANT, DTYPE, [dict(dtype=2)]),
    ("gmm_quantize_int4", QUANT, SHAPE, [dict(group=16), dict(group=256), dict(k=0), dict(k=96), dict(ld=255),
                                         dict(rows=-1), dict(batch=-1), dict(batch=64, rows=LARGEST),
                                         dict(rows=LARGEST + 1), dict(k=LARGEST + 32, ld=LARGEST + 32)]),
    ("gmm_quantize_int4", QUANT, ALIGN, [dict(codes=ODD8), dict(scale=ODD8), dict(zero=ODD), dict(dtype=1, x=ODD)]),
    ("gmm_dequantize_int4", DEQUANT, NULL, [dict(codes=None), dict(scale=None), dict(out=None)]),
    ("gmm_dequantize_int4", DEQUANT, DTYPE, [dict(dtype=2)]),
    ("gmm_dequantize_int4", DEQUANT, SHAPE, [dict(group=48), dict(k=96)]),
    ("gmm_dequantize_int4", DEQUANT, ALIGN, [dict(codes=ODD), dict(scale=ctypes.c_void_p(4097)), dict(dtype=1, out=ODD)]),
    ("gmm_matvec_int4", VEC, NULL, [dict(x=None), dict(codes=None), dict(scale=None), dict(out=None)]),
    ("gmm_matvec_int4", VEC, DTYPE, [dict(out_dtype=2)]),
    ("gmm_matvec_int4", VEC, SHAPE, [dict(tokens=-1), dict(k=0), dict(k=96), dict(n=0), dict(n=12), dict(group=16),
                                     dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=33),
                                     dict(chosen=None), dict(act=3), dict(act=1, n=24), dict(act=1, weights=P),
                                     dict(ld=255), dict(ld=260), dict(k=LARGEST + 1024, ld=LARGEST + 1024),
                                     dict(n=LARGEST + 8), dict(tokens=LARGEST + 1)]),
    ("gmm_matvec_int4", VEC, ALIGN, [dict(x=ODD8), dict(codes=ODD8), dict(scale=ODD8), dict(zero=ODD8), dict(chosen=ODD),
                                     dict(weights=ODD), dict(out_dtype=1, out=ODD), dict(scratch=ODD8)]),
    ("gmm_matvec_int4", VEC, WORKSPACE, [dict(tokens=100, k=4096, ld=4096), dict(tokens=100, k=4096, ld=4096, scratch=P,
                                                                                 scratch_bytes=1000),
                                         dict(tokens=100, k=4096, ld=4096, scratch_bytes=1 << 30)]),
]


@pytest.mark.parametrize("name,base,status,over", [(n, b, s, o) for n, b, s, os_ in REFUSALS for o in os_])
def test_refusals(lib, name, base, status, over):
    assert getattr(lib, name)(*{**base, **over}.values()) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are no memory")
@pytest.mark.parametrize("name,base", [("gmm_balance_loss", LOSS), ("gmm_balance_loss_backward", LBACK),
                                       ("gmm_gated_act", ACT), ("gmm_gated_act_backward", ABACK),
                                       ("gmm_quantize_int4", QUANT), ("gmm_dequantize_int4", DEQUANT),
                                       ("gmm_matvec_int4", VEC)])
def test_good_arguments_reach_the_device_check(lib, name, base):
    assert getattr(lib, name)(*base.values()) in (ARCH, CUDA)


def test_scratch_bytes(lib):
    for tokens, experts, sequences in [(0, 1, 2), (4, 1, 2), (4096, 128, 1), (4096, 128, 4096), (2 ** 30, 1024, 1)]:
        assert lib.gmm_balance_scratch_bytes(tokens, experts, sequences) > 0
    assert lib.gmm_balance_scratch_bytes(192, 8, 1) == 0
    for bad in [(-1, 8, 1), (8, 0, 1), (8, 1025, 1), (8, 8, 0), (8, 8, 3)]:
        assert lib.gmm_balance_scratch_bytes(*bad) == 0


def test_matvec_scratch_bytes(lib):
    assert lib.gmm_matvec_scratch_bytes(1, 4096, 128, 0, 8, 0) == 0
    many = lib.gmm_matvec_scratch_bytes(64, 4096, 128, 0, 4, 0)
    assert many == 64 * (4096 * 2 + 32 * 4 + 4) and lib.gmm_matvec_scratch_bytes(6400, 4096, 128, 0, 4, 0) == many
    for bad in [(0, 4096, 128, 0, 8, 0), (-1, 4096, 128, 0, 8, 0), (64, 0, 128, 0, 8, 0), (64, 4096, 16, 0, 8, 0),
                (64, 4096, 128, 0, 0, 0), (64, 4096, 128, 0, 33, 0)]:
        assert lib.gmm_matvec_scratch_bytes(*bad) == 0


# ---------------------------------------------------------------- the binding, on tensors without memory
I32, U8, F32, BF16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16


@pytest.fixture
def current(monkeypatch):
    monkeypatch.setattr(G, "_current_device", lambda: 0)


def int4(z, name="w", lead=(8,), n=32, k=256, group=64, zero_points=False, **over):
    shape = (*lead, -(-k // 256), n, 256 // group)
    parts = dict(codes=z(f"{name}.codes", (*lead, n, k // 2), U8), scale=z(f"{name}.scale", shape, BF16),
                 zero=z(f"{name}.zero", shape, U8) if zero_points else None, group=group)
    return G.Int4Tensor(**{**parts, **over})


def loss(z, **over):
    parts = dict(losses=z("losses", (2,)), counts=z("balance.counts", (2, 8), I32), tokens=z("balance.tokens", (1,), I32))
    return G.BalanceLoss(**{**parts, **over})


CALLS = {
    "balance_loss": (lambda z: G.balance_loss(z("logits", (4, 8)), z("experts", (4, 2), I32), sequences=2,
                                              token_mask=z("token_mask", (4,), torch.bool)),
                     ["logits", "experts", "token_mask"]),
    "balance_loss_backward": (lambda z: G.balance_loss_backward(z("dlosses", (2,)), loss(z), z("logits", (4, 8)),
                                                                token_mask=z("token_mask", (4,), U8)),
                              ["dlosses", "balance.counts", "balance.tokens", "logits", "token_mask"]),
    "gated_act": (lambda z: G.gated_act(z("h", (4, 16))), ["h"]),
    "gated_act_backward": (lambda z: G.gated_act_backward(z("dout", (4, 8)), z("h", (4, 16))), ["dout", "h"]),
    "quantize_int4": (lambda z: G.quantize_int4(z("x", (4, 256))), ["x"]),
    "quantize_int4 batch": (lambda z: G.quantize_int4(z("x", (2, 4, 256))), ["x"]),
    "dequantize_int4": (lambda z: G.dequantize_int4(int4(z, "q", (), zero_points=True)), ["q.codes", "q.scale", "q.zero"]),
    "matvec_int4": (lambda z: G.matvec_int4(z("x", (4, 256), BF16), int4(z, zero_points=True), z("experts", (4, 2), I32),
                                            z("weights", (4, 2))),
                    ["x", "w.codes", "w.scale", "w.zero", "experts", "weights"]),
    "matvec_int4 slots": (lambda z: G.matvec_int4(z("x", (4, 2, 256), BF16), int4(z), z("experts", (4, 2), I32)),
                          ["x", "experts"]),
    "matvec_int4 dense": (lambda z: G.matvec_int4(z("x", (4, 256), BF16), int4(z, lead=())), ["x", "w.codes"]),
}


@pytest.mark.parametrize("name,operand", [(n, o) for n, (_, operands) in CALLS.items() for o in [*operands, "all"]])
def test_a_tensor_of_another_device_is_refused(current, name, operand):
    with FakeTensorMode():
        def z(what, shape, dtype=F32):
            return torch.empty(shape, dtype=dtype, device="cuda:1" if operand in (what, "all") else "cuda:0")

        with pytest.raises(ValueError, match="is on cuda:1, but the current device is cuda:0") as e:
            CALLS[name][0](z)
    assert operand == "all" or str(e.value).startswith(operand + " ")


def t(*shape, dtype=F32, device="cuda:0"):
    return torch.empty(shape, dtype=dtype, device=device)


def z(what, shape, dtype=F32):
    return t(*shape, dtype=dtype)


def x(*shape):
    return t(*shape, dtype=BF16)


def i(*shape):
    return t(*shape, dtype=I32)


BAD = {
    "balance host": (ValueError, lambda: G.balance_loss(t(4, 8, device="cpu"), i(4, 2))),
    "balance half": (TypeError, lambda: G.balance_loss(t(4, 8).half(), i(4, 2))),
    "balance columns": (ValueError, lambda: G.balance_loss(t(8, 4).t(), i(4, 2))),
    "balance 1-d experts": (ValueError, lambda: G.balance_loss(t(4, 8), i(8))),
    "balance experts' type": (TypeError, lambda: G.balance_loss(t(4, 8), i(4, 2).long())),
    "balance experts' tokens": (ValueError, lambda: G.balance_loss(t(4, 8), i(3, 2))),
    "balance sequences": (ValueError, lambda: G.balance_loss(t(4, 8), i(4, 2), sequences=3)),
    "balance no sequences": (ValueError, lambda: G.balance_loss(t(4, 8), i(4, 2), sequences=0)),
    "balance score": (ValueError, lambda: G.balance_loss(t(4, 8), i(4, 2), "tanh")),
    "balance mask type": (TypeError, lambda: G.balance_loss(t(4, 8), i(4, 2), token_mask=t(4))),
    "balance mask length": (ValueError, lambda: G.balance_loss(t(4, 8), i(4, 2), token_mask=t(5, dtype=torch.bool))),
    "backward counts": (ValueError, lambda: G.balance_loss_backward(t(2), loss(z, counts=i(2, 7)), t(4, 8))),
    "backward sequences": (ValueError, lambda: G.balance_loss_backward(t(2), loss(z, counts=i(3, 8)), t(4, 8))),
    "backward no counts": (ValueError, lambda: G.balance_loss_backward(t(2), loss(z, counts=i(0, 8)), t(4, 8))),
    "backward dlosses": (ValueError, lambda: G.balance_loss_backward(t(3), loss(z), t(4, 8))),
    "backward dlosses type": (TypeError, lambda: G.balance_loss_backward(t(2).double(), loss(z), t(4, 8))),
    "act odd": (ValueError, lambda: G.gated_act(t(4, 15))),
    "act none": (ValueError, lambda: G.gated_act(t(4, 0))),
    "act kind": (ValueError, lambda: G.gated_act(t(4, 16), "relu")),
    "act type": (TypeError, lambda: G.gated_act(t(4, 16).double())),
    "act strided": (ValueError, lambda: G.gated_act(t(4, 32)[:, ::2])),
    "act overlapping": (ValueError, lambda: G.gated_act(t(1, 16).expand(4, 16))),
    "act gradient's type": (TypeError, lambda: G.gated_act_backward(x(4, 8), t(4, 16))),
    "act gradient's size": (ValueError, lambda: G.gated_act_backward(t(4, 16), t(4, 16))),
    "quantize group": (ValueError, lambda: G.quantize_int4(t(4, 256), 16)),
    "quantize k": (ValueError, lambda: G.quantize_int4(t(4, 96), 64)),
    "quantize k 0": (ValueError, lambda: G.quantize_int4(t(4, 0), 64)),
    "quantize 1-d": (ValueError, lambda: G.quantize_int4(t(256))),
    "quantize strided batch": (ValueError, lambda: G.quantize_int4(t(2, 4, 512)[..., :256])),
    "quantize type": (TypeError, lambda: G.quantize_int4(t(4, 256).half())),
    "dequantize scale": (ValueError, lambda: G.dequantize_int4(int4(z, scale=x(8, 1, 32, 2)))),
    "dequantize scale's type": (TypeError, lambda: G.dequantize_int4(int4(z, scale=t(8, 1, 32, 4)))),
    "dequantize zero": (ValueError, lambda: G.dequantize_int4(int4(z, zero=t(8, 1, 32, 2, dtype=U8)))),
    "dequantize zero's type": (TypeError, lambda: G.dequantize_int4(int4(z, zero=t(8, 1, 32, 4)))),
    "dequantize out": (TypeError, lambda: G.dequantize_int4(int4(z), torch.float16)),
    "dequantize codes": (ValueError, lambda: G.dequantize_int4(int4(z, codes=t(32 * 128, dtype=U8)))),
    "matvec k": (ValueError, lambda: G.matvec_int4(x(4, 128), int4(z), i(4, 2))),
    "matvec type": (TypeError, lambda: G.matvec_int4(t(4, 256), int4(z), i(4, 2))),
    "matvec pitch": (ValueError, lambda: G.matvec_int4(x(4, 260)[:, :256], int4(z), i(4, 2))),
    "matvec n": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z, n=12), i(4, 2))),
    "matvec act n": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z, n=24), i(4, 2), act="silu")),
    "matvec act": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 2), act="relu")),
    "matvec act and weights": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 2), t(4, 2), act="silu")),
    "matvec weights alone": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z, lead=()), weights=t(4, 1))),
    "matvec weights' type": (TypeError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 2), x(4, 2))),
    "matvec batch without experts": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z))),
    "matvec experts without batch": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z, lead=()), i(4, 2))),
    "matvec slots without experts": (ValueError, lambda: G.matvec_int4(x(4, 2, 256), int4(z, lead=()))),
    "matvec experts' type": (TypeError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 2).long())),
    "matvec tokens": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z), i(3, 2))),
    "matvec topk 33": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 33))),
    "matvec topk 0": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 0))),
    "matvec slots": (ValueError, lambda: G.matvec_int4(x(4, 3, 256), int4(z), i(4, 2))),
    "matvec strided slots": (ValueError, lambda: G.matvec_int4(x(4, 2, 512)[..., :256], int4(z), i(4, 2))),
    "matvec out": (TypeError, lambda: G.matvec_int4(x(4, 256), int4(z), i(4, 2), out_dtype=torch.float16)),
    "matvec group": (ValueError, lambda: G.matvec_int4(x(4, 256), int4(z, group=16), i(4, 2))),
}


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_tensors_are_refused(current, name):
    error, call = BAD[name]
    real = torch.Tensor.data_ptr
    with FakeTensorMode():
        torch.Tensor.data_ptr = lambda self: 1 << 20  # a fake tensor's is refused by PyTorch
        try:
            with pytest.raises(error):
                call()
        finally:
            torch.Tensor.data_ptr = real
