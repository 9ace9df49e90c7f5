"""The operators of include/libgmm_moe.h: exported, bound, and refusing bad host-side arguments
before anything touches a device (no GPU needed)."""

import ctypes
import os
import re

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "libgmm_moe.h")
P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 2)
NULL, DTYPE, SHAPE, ALIGN, OFFSET, WORKSPACE, ARCH = 1, 2, 3, 4, 5, 6, 7


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load_library()


def test_every_declared_call_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^int\s+(gmm_[a-z0-9_]+)\s*\(", text, flags=re.M)
    assert len(names) == 9
    for name in names:
        assert hasattr(lib, name) and name in G.SIGNATURES
        args = re.search(re.escape(name) + r"\s*\((.*?)\);", text, flags=re.S).group(1)
        assert len(args.split(",")) == len(G.SIGNATURES[name][0]), name


def call(lib, name, defaults, **over):
    return getattr(lib, name)(*{**defaults, **over}.values())


ROUTE = dict(logits=P, dtype=1, tokens=4, experts=8, ld=8, topk=2, score=0, renorm=1, scale=1.0, bias=None, mask=None,
             weights=P, chosen=P, stream=None)
BACK = dict(dweights=P, chosen=P, logits=P, dtype=1, tokens=4, experts=8, ld=8, topk=2, score=0, renorm=1, scale=1.0,
            dlogits=P, stream=None)
SORT = dict(experts=P, tokens=4, topk=2, num=8, sizes=P, rows=P, source=P, stream=None)
DISPATCH = dict(x=P, dtype=0, tokens=4, d=8, ld=8, topk=2, rows=P, source=P, out=P, stream=None)
COMBINE = dict(rows_in=P, dtype=0, tokens=4, d=8, topk=2, rows=P, weights=P, out=P, stream=None)
CBACK = dict(dout=P, rows_in=P, dtype=0, tokens=4, d=8, topk=2, rows=P, source=P, weights=P, din=P, dw=P, stream=None)
QUANT = dict(x=P, dtype=0, batch=1, n=4, k=64, ld=64, fmt=0, rows=None, source=None, topk=1, codes=P, scale=P, row=P,
             stream=None)
DEQUANT = dict(codes=P, scale=P, row=P, fmt=0, batch=1, n=4, k=64, out=P, dtype=0, stream=None)
FP4 = dict(lc=P, ls=P, lr=P, m=4, k=64, rc=P, rs=P, rr=P, fmt=0, local=2, n=16, sizes=P, total=4, offset=0, bias=None,
           bias_dtype=0, out=P, out_dtype=0, ws=P, ws_bytes=256, stream=None)
BIG = 2 ** 31

REFUSALS = [
    ("gmm_route", ROUTE, NULL, [dict(logits=None), dict(weights=None), dict(chosen=None)]),
    ("gmm_route", ROUTE, DTYPE, [dict(dtype=2)]),
    ("gmm_route", ROUTE, SHAPE, [dict(tokens=-1), dict(experts=0), dict(experts=1025, ld=1025), dict(ld=7),
                                 dict(topk=0), dict(topk=9), dict(topk=33, experts=64, ld=64), dict(score=2)]),
    ("gmm_route", ROUTE, ALIGN, [dict(logits=ODD), dict(bias=ODD), dict(weights=ODD), dict(chosen=ODD)]),
    ("gmm_route_backward", BACK, NULL, [dict(dweights=None), dict(chosen=None), dict(logits=None), dict(dlogits=None)]),
    ("gmm_route_backward", BACK, SHAPE, [dict(topk=9), dict(ld=7)]),
    ("gmm_route_backward", BACK, ALIGN, [dict(dlogits=ODD), dict(dweights=ODD)]),
    ("gmm_sort_by_expert", SORT, NULL, [dict(experts=None), dict(sizes=None), dict(rows=None), dict(source=None),
                                        dict(tokens=0, sizes=None)]),
    ("gmm_sort_by_expert", SORT, SHAPE, [dict(num=0), dict(num=1025), dict(topk=0), dict(topk=33), dict(tokens=-1),
                                         dict(tokens=2 ** 30), dict(tokens=2 ** 31 - 1023, topk=1)]),
    ("gmm_sort_by_expert", SORT, ALIGN, [dict(experts=ODD), dict(rows=ODD)]),
    ("gmm_dispatch", DISPATCH, NULL, [dict(x=None), dict(rows=None), dict(source=None), dict(out=None)]),
    ("gmm_dispatch", DISPATCH, DTYPE, [dict(dtype=2)]),
    ("gmm_dispatch", DISPATCH, SHAPE, [dict(d=0), dict(ld=7), dict(topk=33), dict(d=BIG, ld=BIG)]),
    ("gmm_dispatch", DISPATCH, ALIGN, [dict(dtype=1, x=ODD), dict(rows=ODD), dict(source=ODD)]),
    ("gmm_combine", COMBINE, NULL, [dict(rows_in=None), dict(rows=None), dict(out=None)]),
    ("gmm_combine", COMBINE, ALIGN, [dict(dtype=1, out=ODD), dict(weights=ODD)]),
    ("gmm_combine_backward", CBACK, NULL, [dict(dout=None), dict(rows_in=None), dict(rows=None), dict(source=None),
                                           dict(weights=None), dict(din=None), dict(dw=None)]),
    ("gmm_combine_backward", CBACK, ALIGN, [dict(dtype=1, din=ODD), dict(dw=ODD)]),
    ("gmm_quantize_fp4", QUANT, NULL, [dict(x=None), dict(codes=None), dict(scale=None), dict(row=None),
                                       dict(rows=P, topk=2)]),
    ("gmm_quantize_fp4", QUANT, DTYPE, [dict(dtype=2), dict(fmt=2)]),
    ("gmm_quantize_fp4", QUANT, SHAPE, [dict(k=0), dict(k=48), dict(ld=63), dict(batch=0), dict(topk=2),
                                        dict(rows=P, source=P, topk=33), dict(rows=P, source=P, batch=2),
                                        dict(n=BIG), dict(rows=P, source=P, topk=2, n=BIG // 2)]),
    ("gmm_quantize_fp4", QUANT, ALIGN, [dict(codes=ODD), dict(scale=ODD), dict(row=ODD), dict(x=ODD, dtype=1)]),
    ("gmm_dequantize_fp4", DEQUANT, NULL, [dict(codes=None), dict(scale=None), dict(row=None), dict(out=None)]),
    ("gmm_dequantize_fp4", DEQUANT, DTYPE, [dict(dtype=2), dict(fmt=-1)]),
    ("gmm_dequantize_fp4", DEQUANT, SHAPE, [dict(k=16), dict(n=-1)]),
    ("gmm_dequantize_fp4", DEQUANT, ALIGN, [dict(out=ODD)]),
    ("gmm_fp4", FP4, NULL, [dict(lc=None), dict(ls=None), dict(rc=None), dict(rs=None), dict(sizes=None),
                            dict(out=None)]),
    ("gmm_fp4", FP4, DTYPE, [dict(fmt=2), dict(out_dtype=2), dict(bias=P, bias_dtype=2)]),
    ("gmm_fp4", FP4, SHAPE, [dict(k=16), dict(k=80), dict(n=12), dict(n=0), dict(m=-1), dict(local=0), dict(local=5),
                             dict(total=1025), dict(m=BIG), dict(m=BIG - 1, n=BIG - 8)]),
    ("gmm_fp4", FP4, OFFSET, [dict(offset=-1), dict(offset=3)]),
    ("gmm_fp4", FP4, ALIGN, [dict(lc=ODD), dict(ls=ODD), dict(rc=ODD), dict(rs=ODD), dict(out=ODD), dict(lr=ODD)]),
    ("gmm_fp4", FP4, WORKSPACE, [dict(ws=None), dict(ws_bytes=255), dict(ws=ODD)]),
]


@pytest.mark.parametrize("name,defaults,status,overs", REFUSALS, ids=[f"{r[0]}-{r[2]}" for r in REFUSALS])
def test_bad_arguments_are_refused(lib, name, defaults, status, overs):
    for over in overs:
        assert call(lib, name, defaults, **over) == status, over


@pytest.mark.parametrize("use", [
    lambda z: G.route(z((4, 8)), 2),
    lambda z: G.route_backward(z((4, 2)), z((4, 2), torch.int32), z((4, 8))),
    lambda z: G.sort_by_expert(z((4, 2), torch.int32), 4),
    lambda z: G.dispatch(z((4, 8)), G.ExpertOrder(z((4,), torch.int32), z((4, 2), torch.int32), z((8,), torch.int32))),
    lambda z: G.combine(z((8, 8)), G.ExpertOrder(z((4,), torch.int32), z((4, 2), torch.int32), z((8,), torch.int32))),
    lambda z: G.quantize_fp4(z((4, 64))),
    lambda z: G.dequantize_fp4(G.Fp4Tensor(z((4, 32), torch.uint8), z((1, 4, 16), torch.uint8), z((4,)), "nvfp4")),
], ids=["route", "route_backward", "sort_by_expert", "dispatch", "combine", "quantize_fp4", "dequantize_fp4"])
def test_host_tensors_are_refused(lib, use):
    with pytest.raises(ValueError, match="CUDA tensor"):
        use(lambda shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype))
