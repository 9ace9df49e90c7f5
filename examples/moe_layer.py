"""A mixture-of-experts layer on libgmm: a training step in bf16 and a serving step in 4 bits.

    python examples/moe_layer.py

The layer routes each token to `topk` experts, each a gated feed-forward network:
    y[t] = sum_j w[t, j] * wo[e] (silu(wg[e] x[t]) * (wu[e] x[t])),  e = experts[t, j]
with wg and wu one weight wi [experts, 2 f, d] and wo [experts, d, f].

Training: route -> sort_by_expert -> dispatch -> gmm -> gated_act -> gmm -> combine, and back through the
gradient of each, with the losses that balance the experts where these are wanted.  Serving: the same
order, the rows quantised on their way to the experts, and the products of 4-bit rows with 4-bit
weights; or weights in 4-bit integers, for few tokens with matvec_int4() without any order, for many
dequantised on the way to the products of the sorted rows.  The router's product is a plain torch operation.
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
        return G.combine(out, order, weights), (x, logits, weights, experts, order, rows, h, act, out, token_mask)

    def balance(self, saved, sequences=1):
        """The router's losses and the experts' loads of a forward(), as a BalanceLoss."""
        return G.balance_loss(saved[1], saved[3], token_mask=saved[9], sequences=sequences)

    def backward(self, dy, saved, balance=None, dlosses=None):
        """Gradients of x and of the weights, as (dx, {"router", "wi", "wo"}), from dy [tokens, d]; with
        balance, those of <dlosses, balance.losses> added, dlosses float32 [2]."""
        x, logits, weights, experts, order, rows, h, act, out, token_mask = saved
        sizes = order.group_sizes
        dout, dweights = G.combine_backward(dy, out, order, weights)
        dact = G.gmm(dout, self.wo, sizes, transpose_rhs=False)  # the weight as it is, read as [g, k, n]
        dwo = G.tgmm(dout, act, sizes)
        dh = G.gated_act_backward(dact, h)
        drows = G.gmm(dh, self.wi, sizes, transpose_rhs=False)
        dwi = G.tgmm(dh, rows, sizes)
        dlogits = G.route_backward(dweights, experts, logits)
        if balance is not None:
            dlogits = dlogits + G.balance_loss_backward(dlosses, balance, logits, token_mask=token_mask)
        dx = G.dispatch_backward(drows, order) + dlogits @ self.router
        return dx, {"router": dlogits.T @ x, "wi": dwi, "wo": dwo}

    @staticmethod
    def _gate(h):
        return G.gated_act(h)

    # ------------------------------------------------------------ serving
    def pack(self, fmt="nvfp4"):
        """Quantises the experts' weights once, for decode(): "nvfp4", "mxfp4", or "int4" or "uint4" (with zero
        points) in groups of 64."""
        if fmt in ("int4", "uint4"):
            self.packed = tuple(G.quantize_int4(w, 64, zero_points=fmt == "uint4") for w in (self.wi, self.wo))
        else:
            self.packed = G.quantize_fp4(self.wi, fmt), G.quantize_fp4(self.wo, fmt)
        return self

    # Tokens up to which matvec_int4() pays against the weights dequantised for the call: 128 tokens take 1.09 ms
    # for 1.00 (2 of 8 experts, d 4096, f 14336), 0.21 for 0.31 (4 of 64, 2048, 1024), 0.48 for 0.59 (8 of 128,
    # 2048, 1024), 256 tokens 2.18 for 1.01, 0.41 for 0.31 and 0.97 for 0.58.
    FEW = 128

    def decode(self, x):
        """y for x, the experts' products in 4 bits."""
        wi, wo = self.packed
        weights, experts = G.route(x @ self.router.T, self.topk)
        integers = isinstance(wi, G.Int4Tensor)
        if integers and x.shape[0] <= self.FEW:
            return G.matvec_int4(G.matvec_int4(x, wi, experts, act="silu"), wo, experts, weights)
        order = G.sort_by_expert(experts, self.experts)
        if integers:
            h = G.gmm(G.dispatch(x, order), G.dequantize_int4(wi), order.group_sizes)
            return G.combine(G.gmm(G.gated_act(h), G.dequantize_int4(wo), order.group_sizes), order, weights)
        rows = G.quantize_fp4(x, wi.format, order=order)
        h = G.gmm_fp4(rows, wi, order.group_sizes)
        act = G.quantize_fp4(self._gate(h), wo.format)
        return G.combine(G.gmm_fp4(act, wo, order.group_sizes), order, weights)


def main():
    layer = MoeLayer(experts=64, d=2048, f=1024, topk=4)
    x = torch.randn((4096, 2048), device="cuda").to(torch.bfloat16)
    y, saved = layer.forward(x)
    balance = layer.balance(saved)
    dlosses = torch.tensor([0.01, 0.001], device="cuda")
    dx, grads = layer.backward(torch.randn_like(y), saved, balance, dlosses)
    print("training step:", tuple(y.shape), tuple(dx.shape), {k: tuple(v.shape) for k, v in grads.items()})
    print("balance loss %.3f, z loss %.3f," % tuple(balance.losses.tolist()), "loads from", int(balance.counts.min()), "to",
          int(balance.counts.max()))
    for fmt in ("nvfp4", "mxfp4"):
        layer.pack(fmt)
        z = layer.decode(x)
        off = (z.float() - y.float()).norm() / y.float().norm()
        print(f"serving step in {fmt}: {tuple(z.shape)}, off from bf16 by {off:.3f}")
    # decoding steps as CUDA graphs: one replay for all of their launches
    for fmt, tokens in (("mxfp4", 64), ("int4", 1)):
        layer.pack(fmt)
        token = torch.randn((tokens, 2048), device="cuda").to(torch.bfloat16)
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
        print(f"decoding step of {out.shape[0]} tokens in {fmt}: {start.elapsed_time(end) * 10:.1f} us")
    if G.read_device_errors() != 0:
        raise RuntimeError("device error flags set")


if __name__ == "__main__":
    main()
