"""The MoE operators on a stream given as an argument, and with arguments that do not take the binding's
short way: the same bits as on the current stream."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same(a, b):
    if isinstance(a, torch.Tensor):
        return torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) and a.dtype == b.dtype
    if isinstance(a, tuple):
        return len(a) == len(b) and all(same(x, y) for x, y in zip(a, b))
    return a == b


@pytest.fixture(scope="module")
def data():
    gen = torch.Generator(device=DEV).manual_seed(0)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    d = dict(logits=normal(300, 24), x=normal(300, 512).to(torch.bfloat16), dy=normal(300, 512).to(torch.bfloat16),
             g=normal(300, 3), bias=normal(24), mask=torch.arange(300, device=DEV) % 7 != 0,
             w=normal(24, 256, 512).to(torch.bfloat16), out_bias=normal(24, 1, 256))
    d["weights"], d["experts"] = G.route(d["logits"], 3, token_mask=d["mask"])
    d["order"] = G.sort_by_expert(d["experts"], 24)
    d["rows"] = G.dispatch(d["x"], d["order"])
    for fmt in ("nvfp4", "mxfp4"):
        d["q" + fmt] = G.quantize_fp4(d["x"], fmt, order=d["order"])
        d["p" + fmt] = G.quantize_fp4(d["w"], fmt)
    torch.cuda.synchronize()
    return d


CALLS = {
    "route": lambda d, **k: G.route(d["logits"], 3, select_bias=d["bias"], token_mask=d["mask"], **k),
    "route_sigmoid": lambda d, **k: G.route(d["logits"], 3, "sigmoid", False, 2.5, **k),
    "route_backward": lambda d, **k: G.route_backward(d["g"], d["experts"], d["logits"], **k),
    "sort_by_expert": lambda d, **k: G.sort_by_expert(d["experts"], 24, **k),
    "dispatch": lambda d, **k: G.dispatch(d["x"], d["order"], **k),
    "dispatch_backward": lambda d, **k: G.dispatch_backward(d["rows"], d["order"], **k),
    "combine": lambda d, **k: G.combine(d["rows"], d["order"], d["weights"], **k),
    "combine_backward": lambda d, **k: G.combine_backward(d["dy"], d["rows"], d["order"], d["weights"], **k),
    "quantize": lambda d, **k: G.quantize_fp4(d["x"], "nvfp4", **k),
    "quantize_order": lambda d, **k: G.quantize_fp4(d["x"], "mxfp4", order=d["order"], **k),
    "dequantize": lambda d, **k: G.dequantize_fp4(d["qnvfp4"], **k),
    "gmm_fp4": lambda d, **k: G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, **k),
    "gmm_fp4_mx": lambda d, **k: G.gmm_fp4(d["qmxfp4"], d["pmxfp4"], d["order"].group_sizes,
                                           out_dtype=torch.float32, **k),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_given_stream(data, name):
    want = CALLS[name](data)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = CALLS[name](data, stream=side)
    side.synchronize()
    assert same(got, want)


def test_arguments_off_the_short_way(data):
    d = data
    assert same(G.route(d["logits"], 3, scale=2), G.route(d["logits"], 3, scale=2.0))
    assert same(G.route(d["logits"], 3, renormalize="yes"), G.route(d["logits"], 3, renormalize=True))
    assert same(G.route(d["logits"], 3, token_mask=d["mask"].to(torch.uint8)), G.route(d["logits"], 3, token_mask=d["mask"]))
    out = torch.empty((900, 256), dtype=torch.bfloat16, device=DEV)
    want = G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes)
    assert G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, out=out) is out
    assert torch.equal(out, want)
    zero = torch.zeros_like(d["out_bias"])
    assert torch.equal(G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, rhs_bias=zero), want)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    assert torch.equal(G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, workspace=ws), want)
    with pytest.raises(ValueError, match="workspace"):
        G.gmm_fp4(d["qnvfp4"], d["pnvfp4"], d["order"].group_sizes, workspace=torch.zeros(256, dtype=torch.uint8))
    batch = G.dequantize_fp4(d["pnvfp4"])
    one = G.Fp4Tensor(d["pnvfp4"].codes[5], d["pnvfp4"].block_scale[5], d["pnvfp4"].row_scale[5], "nvfp4")
    assert torch.equal(G.dequantize_fp4(one), batch[5])


def test_four_bit_weights_serve_the_bf16_product_too(data):
    """NVFP4 weights packed here are gmm()'s microscaled weights once their scales are put in row order."""
    d = data
    p = d["pnvfp4"]
    scales = p.block_scale.permute(0, 2, 1, 3).reshape(24, 256, -1)[:, :, : 512 // 16].contiguous()
    out = G.gmm(d["rows"], p.codes, d["order"].group_sizes, rhs_scale=p.row_scale.view(24, 1, 1, 256),
                rhs_format="e2m1", rhs_block_scale=scales.view(torch.float8_e4m3fn), out_dtype=torch.float32)
    w = G.dequantize_fp4(p, torch.float32).double()
    at = 0
    for g, size in enumerate(d["order"].group_sizes.tolist()):
        a = d["rows"][at:at + size].double()
        ref, mag = a @ w[g].T, a.abs() @ w[g].abs().T
        assert ((out[at:at + size].double() - ref).abs() <= 1e-3 * mag).all()
        at += size
