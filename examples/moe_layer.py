"""A mixture-of-experts layer on libgmm: a training step in bf16 and a serving step in 4 bits.

    python examples/moe_layer.py

The layer routes each token to `topk` experts, each a gated feed-forward network:
    y[t] = sum_j w[t, j] * wo[e] (silu(wg[e] x[t]) * (wu[e] x[t])),  e = experts[t, j]
with wg and wu one weight wi [experts, 2 f, d] and wo [experts, d, f].

Training: route -> sort_by_expert -> dispatch -> gmm -> gmm -> combine, and back through the gradient
of each.  Serving: the same order, the rows quantised on their way to the experts, and the products of
4-bit rows with 4-bit weights.  The router's product and the activation are plain torch operations.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_matrix_gb300 as G  # noqa: E402


class MoeLayer:
    def __init__(self, experts, d, f, topk, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, generator=gen, device=device) / shape[-1] ** 0.5
            return w.to(torch.bfloat16)

        self.topk, self.experts = topk, experts
        self.router = weight(experts, d)
        self.wi, self.wo = weight(experts, 2 * f, d), weight(experts, d, f)
        self.packed = None

    # ------------------------------------------------------------ training
    def forward(self, x, token_mask=None):
        """y [tokens, d] for x [tokens, d] bf16, and what backward() needs."""
        logits = x @ self.router.T
        weights, experts = G.route(logits, self.topk, token_mask=token_mask)
        order = G.sort_by_expert(experts, self.experts)
        rows = G.dispatch(x, order)
        h = G.gmm(rows, self.wi, order.group_sizes)
        act = self._gate(h)
        out = G.gmm(act, self.wo, order.group_sizes)
        return G.combine(out, order, weights), (x, logits, weights, experts, order, rows, h, act, out)

    def backward(self, dy, saved):
        """Gradients of x and of the weights, as (dx, {"router", "wi", "wo"}), from dy [tokens, d]."""
        x, logits, weights, experts, order, rows, h, act, out = saved
        sizes = order.group_sizes
        dout, dweights = G.combine_backward(dy, out, order, weights)
        dact = G.gmm(dout, self.wo, sizes, transpose_rhs=False)  # the weight as it is, read as [g, k, n]
        dwo = G.tgmm(dout, act, sizes)
        gate, up = h.float().chunk(2, dim=1)
        s = torch.sigmoid(gate)
        d = dact.float()
        dh = torch.cat((d * up * s * (1 + gate * (1 - s)), d * gate * s), dim=1).to(torch.bfloat16)
        drows = G.gmm(dh, self.wi, sizes, transpose_rhs=False)
        dwi = G.tgmm(dh, rows, sizes)
        dlogits = G.route_backward(dweights, experts, logits)
        dx = G.dispatch_backward(drows, order) + dlogits @ self.router
        return dx, {"router": dlogits.T @ x, "wi": dwi, "wo": dwo}

    @staticmethod
    def _gate(h):
        gate, up = h.float().chunk(2, dim=1)
        return (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)

    # ------------------------------------------------------------ serving
    def pack(self, fmt="nvfp4"):
        """Quantises the experts' weights once, for decode()."""
        self.packed = G.quantize_fp4(self.wi, fmt), G.quantize_fp4(self.wo, fmt)
        return self

    def decode(self, x):
        """y for x, the experts' products in 4 bits."""
        wi, wo = self.packed
        weights, experts = G.route(x @ self.router.T, self.topk)
        order = G.sort_by_expert(experts, self.experts)
        rows = G.quantize_fp4(x, wi.format, order=order)
        h = G.gmm_fp4(rows, wi, order.group_sizes)
        act = G.quantize_fp4(self._gate(h), wo.format)
        return G.combine(G.gmm_fp4(act, wo, order.group_sizes), order, weights)


def main():
    layer = MoeLayer(experts=64, d=2048, f=1024, topk=4)
    x = torch.randn((4096, 2048), device="cuda").to(torch.bfloat16)
    y, saved = layer.forward(x)
    dx, grads = layer.backward(torch.randn_like(y), saved)
    print("training step:", tuple(y.shape), tuple(dx.shape), {k: tuple(v.shape) for k, v in grads.items()})
    for fmt in ("nvfp4", "mxfp4"):
        layer.pack(fmt)
        z = layer.decode(x)
        off = (z.float() - y.float()).norm() / y.float().norm()
        print(f"serving step in {fmt}: {tuple(z.shape)}, off from bf16 by {off:.3f}")
    # a decoding step as a CUDA graph: one replay for all of its launches
    token = torch.randn((64, 2048), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(token)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = layer.decode(token)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"decoding step of {out.shape[0]} tokens: {start.elapsed_time(end) * 10:.1f} us")
    if G.read_device_errors() != 0:
        raise RuntimeError("device error flags set")


if __name__ == "__main__":
    main()
