"""How the operators of include/libgmm_experts.h are called: on the current or a given stream, by either way of
the binding, under a dispatch mode, in CUDA graphs, two at once; the same bits each time."""

import pytest
import torch

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import moe
from test_dispatch_modes_gpu import Allocations
from test_moe_streams_gpu import DEV, same
from test_stream_results_gpu import pool_of, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def data():
    gen = torch.Generator(device=DEV).manual_seed(0)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=DEV).to(dtype)

    d = dict(logits=normal(300, 24), mask=torch.arange(300, device=DEV) % 7 != 0, h=normal(300, 1024), dout=normal(300, 512),
             x=normal(9, 512), slots=normal(9, 3, 512), w=normal(24, 256, 512), dlosses=torch.tensor([0.1, 0.01], device=DEV),
             f32=normal(70, 320, dtype=torch.float32))
    d["weights"], d["experts"] = G.route(d["logits"], 3, token_mask=d["mask"])
    d["few"], d["few_weights"] = d["experts"][1:10].contiguous(), d["weights"][1:10].contiguous()
    d["loss"] = G.balance_loss(d["logits"], d["experts"], sequences=4)
    d["q"], d["qz"] = G.quantize_int4(d["w"]), G.quantize_int4(d["w"], 32, True)
    d["one"] = G.Int4Tensor(d["q"].codes[2], d["q"].scale[2], None, 128)
    d["rows"] = G.quantize_int4(d["f32"], 64, True)
    torch.cuda.synchronize()
    return d


CALLS = {
    "balance_loss": lambda d, **k: G.balance_loss(d["logits"], d["experts"], sequences=4, **k),
    "balance_loss_mask": lambda d, **k: G.balance_loss(d["logits"], d["experts"], "sigmoid", d["mask"], **k),
    "balance_loss_backward": lambda d, **k: G.balance_loss_backward(d["dlosses"], d["loss"], d["logits"], **k),
    "gated_act": lambda d, **k: G.gated_act(d["h"], **k),
    "gated_act_backward": lambda d, **k: G.gated_act_backward(d["dout"], d["h"], "gelu", **k),
    "quantize_int4": lambda d, **k: G.quantize_int4(d["f32"], 64, True, **k),
    "quantize_int4_batch": lambda d, **k: G.quantize_int4(d["w"], **k),
    "dequantize_int4": lambda d, **k: G.dequantize_int4(d["rows"], torch.float32, **k),
    "dequantize_int4_batch": lambda d, **k: G.dequantize_int4(d["q"], **k),
    "matvec_int4": lambda d, **k: G.matvec_int4(d["x"], d["qz"], d["few"], **k),
    "matvec_int4_act": lambda d, **k: G.matvec_int4(d["x"], d["q"], d["few"], act="silu", out_dtype=torch.float32, **k),
    "matvec_int4_sum": lambda d, **k: G.matvec_int4(d["slots"], d["q"], d["few"], d["few_weights"], **k),
    "matvec_int4_one": lambda d, **k: G.matvec_int4(d["x"], d["one"], **k),
}
RESULTS = {"balance_loss": 4, "balance_loss_mask": 3, "quantize_int4": 3, "quantize_int4_batch": 2}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_given_stream(data, name):
    want = CALLS[name](data)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = CALLS[name](data, stream=side)
    side.synchronize()
    assert same(got, want)
    segments = torch.cuda.memory_snapshot()
    assert all(pool_of(t, segments) == side.cuda_stream for t in tensors(got))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_current_stream(data, name):
    want = CALLS[name](data)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = CALLS[name](data)
    side.synchronize()
    segments = torch.cuda.memory_snapshot()
    assert same(got, want) and all(pool_of(t, segments) == side.cuda_stream for t in tensors(got))


def outcome(call):
    try:
        return call(), None
    except (TypeError, ValueError, RuntimeError) as e:
        return None, (type(e), str(e))


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def i(*shape):
    return t(*shape, dtype=torch.int32)


def x(*shape):
    return t(*shape, dtype=torch.bfloat16)


def int4(*lead, n=32, k=256, group=64, **over):
    parts = dict(codes=t(*lead, n, k // 2, dtype=torch.uint8), scale=x(*lead, -(-k // 256), n, 256 // group), zero=None,
                 group=group)
    return G.Int4Tensor(**{**parts, **over})


class Odd(torch.Tensor):
    pass


ARGUMENTS = {
    "balance topk 33": lambda: G.balance_loss(t(4, 64), i(4, 33)),
    "balance no slots": lambda: G.balance_loss(t(4, 8), i(4, 0)),
    "balance 1025": lambda: G.balance_loss(t(4, 1025), i(4, 2)),
    "balance no experts": lambda: G.balance_loss(t(4, 0), i(4, 2)),
    "balance sequences": lambda: G.balance_loss(t(4, 8), i(4, 2), sequences=3),
    "balance float sequences": lambda: G.balance_loss(t(4, 8), i(4, 2), sequences=2.0),
    "balance score": lambda: G.balance_loss(t(4, 8), i(4, 2), "tanh"),
    "balance pitch": lambda: G.balance_loss(t(4, 16)[:, :8], i(4, 2)),
    "balance every other": lambda: G.balance_loss(t(4, 16)[:, ::2], i(4, 2)),
    "balance subclass": lambda: G.balance_loss(t(4, 8).as_subclass(Odd), i(4, 2)),
    "balance parameter": lambda: G.balance_loss(torch.nn.Parameter(t(4, 8)), i(4, 2)),
    "balance mask": lambda: G.balance_loss(t(4, 8), i(4, 2), token_mask=t(4, dtype=torch.uint8)),
    "balance mask length": lambda: G.balance_loss(t(4, 8), i(4, 2), token_mask=t(5, dtype=torch.bool)),
    "act odd": lambda: G.gated_act(t(4, 15)),
    "act kind": lambda: G.gated_act(t(4, 16), "relu"),
    "act 1-d": lambda: G.gated_act(t(16)),
    "act one row": lambda: G.gated_act(t(1, 16).expand(1, 16)),
    "act pitch": lambda: G.gated_act(t(4, 32)[:, 3:19]),
    "act half": lambda: G.gated_act(t(4, 16).half()),
    "act gradient's type": lambda: G.gated_act_backward(x(4, 8), t(4, 16)),
    "quantize group": lambda: G.quantize_int4(t(4, 256), 48),
    "quantize float group": lambda: G.quantize_int4(t(4, 256), 64.0),
    "quantize k": lambda: G.quantize_int4(t(4, 96), 64),
    "quantize yes": lambda: G.quantize_int4(t(4, 256), 64, "yes"),
    "quantize expanded": lambda: G.quantize_int4(t(1, 256).expand(4, 256)),
    "quantize empty": lambda: G.quantize_int4(t(0, 256)),
    "quantize no columns": lambda: G.quantize_int4(t(4, 0)),
    "dequantize scale": lambda: G.dequantize_int4(int4(scale=x(1, 32, 3))),
    "dequantize zero": lambda: G.dequantize_int4(int4(zero=x(1, 32, 4))),
    "dequantize out": lambda: G.dequantize_int4(int4(), torch.float16),
    "dequantize group": lambda: G.dequantize_int4(int4(group=128)._replace(group=96)),
    "matvec": lambda: G.matvec_int4(x(4, 256), int4(3), i(4, 2)),
    "matvec k": lambda: G.matvec_int4(x(4, 128), int4(3), i(4, 2)),
    "matvec f32": lambda: G.matvec_int4(t(4, 256), int4(3), i(4, 2)),
    "matvec n": lambda: G.matvec_int4(x(4, 256), int4(3, n=12), i(4, 2)),
    "matvec n act": lambda: G.matvec_int4(x(4, 256), int4(3, n=24), i(4, 2), act="silu"),
    "matvec no rows": lambda: G.matvec_int4(x(4, 256), int4(3, n=0), i(4, 2)),
    "matvec no experts": lambda: G.matvec_int4(x(4, 256), int4(0), i(4, 2)),
    "matvec 1025": lambda: G.matvec_int4(x(4, 256), int4(1025, n=8), i(4, 2)),
    "matvec pitch": lambda: G.matvec_int4(x(4, 264)[:, :256], int4(3), i(4, 2)),
    "matvec odd pitch": lambda: G.matvec_int4(x(4, 257)[:, :256], int4(3), i(4, 2)),
    "matvec not aligned": lambda: G.matvec_int4(x(4, 264)[:, 4:260], int4(3), i(4, 2)),
    "matvec slots": lambda: G.matvec_int4(x(4, 2, 256), int4(3), i(4, 2), t(4, 2)),
    "matvec other slots": lambda: G.matvec_int4(x(4, 3, 256), int4(3), i(4, 2)),
    "matvec weights": lambda: G.matvec_int4(x(4, 256), int4(3), i(4, 2), t(4, 3)),
    "matvec weights and act": lambda: G.matvec_int4(x(4, 256), int4(3), i(4, 2), t(4, 2), "silu"),
    "matvec out": lambda: G.matvec_int4(x(4, 256), int4(3), i(4, 2), out_dtype=torch.float16),
    "matvec tokens": lambda: G.matvec_int4(x(4, 256), int4(3), i(5, 2)),
    "matvec empty": lambda: G.matvec_int4(x(0, 256), int4(3), i(0, 2)),
    "matvec topk 33": lambda: G.matvec_int4(x(4, 256), int4(3), i(4, 33)),
}


@pytest.mark.parametrize("name", sorted(CALLS) + sorted(ARGUMENTS))
def test_both_ways_agree(data, name, monkeypatch):
    call = ARGUMENTS[name] if name in ARGUMENTS else lambda: CALLS[name](data)
    short = outcome(call)
    assert not isinstance(moe._calls or moe._bind(), moe._NoCalls)
    monkeypatch.setattr(moe, "_calls", moe._NoCalls())
    long = outcome(call)
    torch.cuda.synchronize()
    assert short[1] == long[1]
    assert short[1] is not None or same(short[0], long[0])


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_mode_sees_the_results(data, name):
    want = CALLS[name](data)
    with Allocations() as seen:
        got = CALLS[name](data)
    assert seen.count == RESULTS.get(name, 1) and same(got, want)


def captured(call, side):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
    with torch.cuda.graph(graph, stream=side):
        got = call()
    return graph, got


@pytest.mark.parametrize("name", sorted(CALLS))
def test_two_graphs_at_once(data, name):
    """Each graph's results and scratch are its own: replayed together on two streams, many times, they agree."""
    want = CALLS[name](data)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    both = [captured(lambda: CALLS[name](data), s) for s in sides]
    torch.cuda.synchronize()
    for _, got in both:
        for r in tensors(got):
            r.fill_(1)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (graph, _) in zip(sides, both):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(got, want) for _, got in both)


def test_new_inputs_in_a_graph(data):
    """A graph of a decoding step's calls follows what is written into its inputs."""
    d = data
    logits, xs = d["logits"][:9].clone(), d["x"].clone()

    def step():
        weights, experts = G.route(logits, 3)
        h = G.matvec_int4(xs, d["q"], experts, act="silu")
        return G.matvec_int4(torch.cat((h, h, h, h), 2), d["qz"], experts, weights), G.balance_loss(logits, experts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, got = captured(step, side)
    for seed in range(3):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        logits.copy_(torch.randn((9, 24), generator=gen, device=DEV))
        xs.copy_(torch.randn((9, 512), generator=gen, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, step())
