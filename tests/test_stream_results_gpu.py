"""Results of calls with stream= are that stream's memory: the allocator hands a freed block out again in
the order of the stream it was allocated on, so a result from another stream's blocks could be written
while that stream still reads what was there, or be given away while the call is still writing it."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from test_moe_streams_gpu import CALLS, DEV, data  # noqa: F401

pytestmark = pytest.mark.gpu

PRODUCTS = {
    "gmm": lambda d, **k: G.gmm(d["rows"], d["w"], d["order"].group_sizes, **k),
    "gmm_options": lambda d, **k: G.gmm(d["rows"], d["w"], d["order"].group_sizes, options={"bf16_kernel": "single"}, **k),
    "tgmm": lambda d, **k: G.tgmm(d["rows"], d["rows"], d["order"].group_sizes, **k),
    "tgmm_local": lambda d, **k: G.tgmm_local(d["rows"], d["rows"], d["order"].group_sizes, 3, 4, **k),
    "quantize_e4m3": lambda d, **k: G.quantize_e4m3(d["rows"], **k),
    "quantize_batch": lambda d, **k: G.quantize_fp4(d["w"], "nvfp4", **k),
    "dequantize_batch": lambda d, **k: G.dequantize_fp4(d["pmxfp4"], **k),
    "gmm_fp4_bias": lambda d, **k: G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, rhs_bias=d["out_bias"], **k),
}


def tensors(x):
    if isinstance(x, torch.Tensor):
        return [x]
    return [t for y in x for t in tensors(y)] if isinstance(x, tuple) else []


def pool_of(t, segments):
    """The stream whose blocks t lies in."""
    for s in segments:
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("name", sorted(CALLS) + sorted(PRODUCTS))
def test_results_are_the_given_streams(data, name):  # noqa: F811
    call = CALLS.get(name) or PRODUCTS[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tensors(call(data, stream=side))
    side.synchronize()
    segments = torch.cuda.memory_snapshot()
    assert got and all(pool_of(t, segments) == side.cuda_stream for t in got)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("name", sorted(CALLS) + sorted(PRODUCTS))
def test_results_are_the_current_streams(data, name):  # noqa: F811
    call = CALLS.get(name) or PRODUCTS[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = tensors(call(data))
        main = tensors(call(data, stream=torch.cuda.default_stream()))
    side.synchronize()
    torch.cuda.synchronize()
    segments = torch.cuda.memory_snapshot()
    assert all(pool_of(t, segments) == side.cuda_stream for t in got)
    assert all(pool_of(t, segments) == torch.cuda.default_stream().cuda_stream for t in main)
