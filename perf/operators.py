"""The operators around the experts' products of a mixture-of-experts layer: what is timed, and their plain forms.

  route     the router's choice of experts for each token and the weights of the choice, with its gradient
  dispatch  the tokens' rows sorted by expert, with the gradient that brings them back
  combine   the experts' rows back in token order, summed with the router's weights, with its gradients
  quantize  rows in microscaled 4-bit floating point (NVFP4 or MXFP4), and the values that they stand for
  product   the grouped product of such rows with such weights, the rows quantised on the way from token order

NVFP4 is e2m1 codes with an e4m3 scale for each 16 of them and a power of two for each row; MXFP4 is e2m1 codes with an
E8M0 scale for each 32.  Scales are stored by windows of k: [.., k / 256 (NVFP4) or k / 512 (MXFP4), rows, 16] bytes.
"""

import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _gmm():
    import moe_grouped_matrix_gb300 as G

    return G


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 64 sequences choosing 4 of 64 experts: all latency
        dict(name="route_decode", op="route", tokens=64, experts=64, topk=4, dtype="f32", score="softmax",
             renormalize=True, biased=False, backward=False),
        # the router of a training step, 8 of 128 experts for 4096 tokens, weights taken from the softmax over all of them
        dict(name="route_train", op="route", tokens=4096, experts=128, topk=8, dtype="bf16", score="softmax",
             renormalize=False, biased=True, backward=True),
        # one decoding step: 256 rows of 4096
        dict(name="dispatch_decode", op="dispatch", tokens=64, experts=64, topk=4, d=4096, dtype="bf16", dropped=0.0,
             backward=False),
        # a training step of a 128-expert layer, with padding tokens that no expert gets
        dict(name="dispatch_train", op="dispatch", tokens=4096, experts=128, topk=8, d=2048, dtype="bf16", dropped=0.05,
             backward=True),
        # one decoding step back in token order
        dict(name="combine_decode", op="combine", tokens=64, experts=64, topk=4, d=2048, dtype="bf16", dropped=0.0,
             backward=False),
        # a training step of an 8-expert layer
        dict(name="combine_train", op="combine", tokens=8192, experts=8, topk=2, d=4096, dtype="bf16", dropped=0.0,
             backward=True),
        # f32 rows of an odd width, some slots dropped
        dict(name="combine_train_f32_odd", op="combine", tokens=3001, experts=61, topk=5, d=1027, dtype="f32",
             dropped=0.1, backward=True),
        # a decoding step's rows
        dict(name="quantize_decode", op="quantize", rows=256, d=4096, dtype="bf16", format="nvfp4"),
        # the rows of a large batch before the experts' first product
        dict(name="quantize_batch", op="quantize", rows=16384, d=4096, dtype="bf16", format="mxfp4"),
        # a decoding step through 64 experts: all the weights are read for 256 rows
        dict(name="product_decode", op="product", tokens=64, experts=64, topk=4, d=4096, n=2048, format="nvfp4",
             out="bf16"),
        # the first product of a 128-expert layer for 4096 tokens, its busiest experts with many times the rows of the others
        dict(name="product_batch", op="product", tokens=4096, experts=128, topk=8, d=2048, n=2048, format="mxfp4",
             out="bf16"),
        # 8 large experts: the up projections of 8192 tokens
        dict(name="product_prefill", op="product", tokens=8192, experts=8, topk=2, d=4096, n=28672, format="nvfp4",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "dispatch", "combine", "quantize", "product"))
    if op == "route":
        experts = _log(rng, 8, 256)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, topk=rng.randint(1, 8),
                    dtype=rng.choice(("bf16", "f32")), score=rng.choice(("softmax", "sigmoid")),
                    renormalize=rng.random() < 0.5, biased=rng.random() < 0.5, backward=rng.random() < 0.5)
    if op in ("dispatch", "combine"):
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=_log(rng, 8, 256), topk=rng.randint(1, 8),
                    d=_log(rng, 64, 2048), dtype=rng.choice(("bf16", "f32")), dropped=rng.choice((0.0, 0.1)),
                    backward=rng.random() < 0.5)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 16384), d=32 * _log(rng, 2, 128), dtype=rng.choice(("bf16", "f32")),
                    format=rng.choice(("nvfp4", "mxfp4")))
    return dict(op=op, tokens=_log(rng, 1, 4096), experts=_log(rng, 8, 64), topk=rng.randint(1, 4),
                d=32 * _log(rng, 8, 128), n=8 * _log(rng, 32, 512), format=rng.choice(("nvfp4", "mxfp4")),
                out=rng.choice(("bf16", "bf16", "f32")))


# ---------------------------------------------------------------- inputs
def _choice(case, gen):
    """Distinct experts for each token, some chosen far more often than others; -1 in the slots that were dropped."""
    T, E, K = case["tokens"], case["experts"], min(case["topk"], case["experts"])
    pull = 0.6 * torch.randn(E, generator=gen, device="cuda")
    score = pull + torch.randn((T, E), generator=gen, device="cuda")
    experts = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32)
    if case.get("dropped"):
        gone = torch.rand((T, K), generator=gen, device="cuda") < case["dropped"]
        experts = torch.where(gone, torch.full_like(experts, -1), experts)
    return experts.contiguous()


def _order(experts, E):
    """The counting sort by expert: sizes of the groups, the row of each slot, the slot of each row (-1: none)."""
    flat = experts.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    slots = torch.sort(key, stable=True)[1]
    sizes = torch.zeros(E + 1, dtype=torch.int32, device=flat.device).scatter_add_(
        0, key, torch.ones_like(key, dtype=torch.int32))[:E]
    at = torch.arange(flat.numel(), device=flat.device)
    kept = at < sizes.sum()
    source = torch.where(kept, slots, torch.full_like(slots, -1)).to(torch.int32)
    rows = torch.empty_like(at).scatter_(0, slots, torch.where(kept, at, torch.full_like(at, -1)))
    return sizes, rows.to(torch.int32).reshape(experts.shape), source


def _pow2(e):
    """2^e in 32 bits for whole -126 <= e <= 127, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _fp4(x, fmt):
    """x [.., k] in 32 bits as (e2m1 codes with their sign bit, block scales as stored, rows' scales, values)."""
    block = BLOCK[fmt]
    six = torch.full((), 6.0, device=x.device)
    a = x.abs()
    fine = torch.isfinite(a)
    bad = ~fine.unflatten(-1, (-1, block)).all(-1)  # a NaN scale, and nothing for the row's
    blocks = a.unflatten(-1, (-1, block)).amax(-1)
    blocks = torch.where(bad, torch.zeros_like(blocks), blocks)
    if fmt == "nvfp4":
        frac, e = torch.frexp(blocks.amax(-1))
        e = (e - 12 + (frac > 0.65625)).clamp(-126, 127)  # the least with amax <= 6 * 448 * 2^e
        e = torch.where(frac == 0, torch.zeros_like(e), e)
        row = _pow2(e)
        down = _pow2(-e.clamp(-126, 126))
        x, blocks = x * down[..., None], blocks * down[..., None]
        s8 = (blocks / six).to(torch.float8_e4m3fn)
        s8 = torch.where(bad, torch.full_like(blocks, math.nan).to(torch.float8_e4m3fn).view(torch.uint8),
                         s8.view(torch.uint8))
        s = s8.view(torch.float8_e4m3fn).float()
    else:
        row = None
        frac, e = torch.frexp(blocks)
        e = (e - 3 + (frac > 0.75)).clamp(-127, 127)  # the least with amax <= 6 * 2^e
        e = torch.where(frac == 0, torch.full_like(e, -127), e)
        s8 = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
        s = torch.where(bad, torch.full_like(blocks, math.nan), _pow2(e.clamp(-126, 127)) * torch.where(e < -126, 0.5, 1.0))
    v = x.abs().unflatten(-1, (-1, block)) / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    code = torch.where(((s > 0) & ~bad)[..., None], code, torch.zeros_like(code))
    table = torch.tensor(E2M1, device=x.device)
    sign = torch.where(bad[..., None], torch.zeros_like(code), torch.signbit(x).unflatten(-1, (-1, block)).to(torch.uint8))
    values = table[code.int()] * (1.0 - 2.0 * sign) * s[..., None]
    values = values.flatten(-2)
    if row is not None:
        values = values * row[..., None]
    return (code + 8 * sign).flatten(-2), s8, row, values


def _windows(s8):
    """Block scales [.., rows, k / block] by windows of 16 of them, [.., windows, rows, 16], zeros past the end."""
    nb = s8.shape[-1]
    w = -(-nb // 16)
    full = torch.zeros(s8.shape[:-1] + (w * 16,), dtype=torch.uint8, device=s8.device)
    full[..., :nb] = s8
    return full.unflatten(-1, (w, 16)).transpose(-3, -2).contiguous()


def _weight_values(codes, scale, row, fmt, k):
    """The values, in 32 bits, of weights [n, k] stored as codes [n, k / 2], scales [windows, n, 16] and rows' scales [n]."""
    both = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    s8 = scale.transpose(0, 1).flatten(1)[:, : k // BLOCK[fmt]]
    if fmt == "nvfp4":
        s = s8.contiguous().view(torch.float8_e4m3fn).float() * row[:, None]
    else:
        s = _pow2(s8.to(torch.int32).clamp(1) - 127) * torch.where(s8 == 0, 0.5, 1.0)
    return (table[both.int()].unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std, dtype=torch.float32):
        return (std * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    op, s = case["op"], dict(case=case)
    if op == "route":
        T, E, K = case["tokens"], case["experts"], min(case["topk"], case["experts"])
        logits = normal((T, E), 1.5, DTYPES[case["dtype"]])
        logits[:, seed % E] = -math.inf  # an expert that is switched off
        mask = torch.rand(T, generator=gen, device="cuda") > 0.03
        mask[0] = True
        logits[~mask] = math.nan  # padding tokens: what is there does not count
        s.update(logits=logits, mask=mask, bias=normal((E,), 0.1) if case["biased"] else None,
                 dweights=normal((T, K), 0.01) if case["backward"] else None)
    elif op == "dispatch":
        T, K, D = case["tokens"], min(case["topk"], case["experts"]), case["d"]
        s.update(experts=_choice(case, gen), x=normal((T, D), 1.0, DTYPES[case["dtype"]]),
                 drows=normal((T * K, D), 0.01, DTYPES[case["dtype"]]) if case["backward"] else None)
    elif op == "combine":
        T, K, D = case["tokens"], min(case["topk"], case["experts"]), case["d"]
        sizes, rows_of, source = _order(_choice(case, gen), case["experts"])
        weights = torch.softmax(normal((T, K), 1.0), dim=1)
        s.update(sizes=sizes, rows_of=rows_of, source=source, weights=weights,
                 rows=normal((T * K, D), 1.0, DTYPES[case["dtype"]]),
                 dout=normal((T, D), 0.01, DTYPES[case["dtype"]]) if case["backward"] else None)
    elif op == "quantize":
        x = normal((case["rows"], case["d"]), 1.0)
        x *= torch.exp(normal((case["rows"], 1), 1.0))  # rows of different sizes
        x[:, seed % case["d"]] *= 30.0  # a channel that stands out
        if case["rows"] > 2:
            x[case["rows"] // 2] = 0.0
        s.update(x=x.to(DTYPES[case["dtype"]]))
    else:
        T, E, D, N = case["tokens"], case["experts"], case["d"], case["n"]
        experts = _choice(case, gen)
        sizes, rows_of, source = _order(experts, E)
        codes = torch.empty((E, N, D // 2), dtype=torch.uint8, device="cuda")
        windows = -(-D // (16 * BLOCK[case["format"]]))
        scale = torch.empty((E, windows, N, 16), dtype=torch.uint8, device="cuda")
        row = torch.empty((E, N), device="cuda") if case["format"] == "nvfp4" else None
        for g in range(E):
            c, s8, r, _ = _fp4(normal((N, D), 0.02), case["format"])
            codes[g] = c[:, 0::2] | (c[:, 1::2] << 4)
            scale[g] = _windows(s8)
            if row is not None:
                row[g] = r
        s.update(sizes=sizes, rows_of=rows_of, source=source, codes=codes, scale=scale, row=row,
                 host_sizes=sizes.tolist(), x=normal((T, D), 1.0, torch.bfloat16))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](s, s["case"])


def _own_route(s, c):
    G = _gmm()
    how = dict(score=c["score"], renormalize=c["renormalize"])
    weights, experts = G.route(s["logits"], min(c["topk"], c["experts"]), select_bias=s["bias"], token_mask=s["mask"], **how)
    out = dict(weights=weights, experts=experts)
    if c["backward"]:
        out["dlogits"] = G.route_backward(s["dweights"], experts, s["logits"], **how)
    return out


def _own_dispatch(s, c):
    G = _gmm()
    order = G.sort_by_expert(s["experts"], c["experts"])
    out = dict(sizes=order.group_sizes, rows_of=order.rows, source=order.source, rows=G.dispatch(s["x"], order))
    if c["backward"]:
        out["dx"] = G.dispatch_backward(s["drows"], order)
    return out


def _own_combine(s, c):
    G = _gmm()
    order = G.ExpertOrder(s["sizes"], s["rows_of"], s["source"])
    out = dict(out=G.combine(s["rows"], order, s["weights"]))
    if c["backward"]:
        out["drows"], out["dweights"] = G.combine_backward(s["dout"], s["rows"], order, s["weights"])
    return out


def _own_quantize(s, c):
    G = _gmm()
    return dict(values=G.dequantize_fp4(G.quantize_fp4(s["x"], c["format"])))


def _own_product(s, c):
    G = _gmm()
    weights = G.Fp4Tensor(s["codes"], s["scale"], s["row"], c["format"])
    rows = G.quantize_fp4(s["x"], c["format"], order=G.ExpertOrder(s["sizes"], s["rows_of"], s["source"]))
    return dict(out=G.gmm_fp4(rows, weights, s["sizes"], out_dtype=DTYPES[c["out"]]))


def _plain_route(s, c):
    K, mask = min(c["topk"], c["experts"]), s["mask"][:, None]
    logits = torch.where(mask, s["logits"].float(), torch.full((), -math.inf, device="cuda"))
    key = logits if s["bias"] is None else logits + s["bias"]
    best, experts = torch.sort(key, dim=1, descending=True, stable=True)
    best, experts = best[:, :K], experts[:, :K]
    took = best > -math.inf
    chosen = torch.where(took, logits.gather(1, experts), torch.zeros_like(best))
    if c["score"] == "sigmoid":
        value = torch.clamp(chosen, max=0.0) - torch.log1p(torch.exp(-chosen.abs()))  # log of the sigmoid
    else:
        value = chosen
    zero = torch.zeros_like(value)
    if c["renormalize"]:
        top = torch.where(took, value, torch.full_like(value, -math.inf)).amax(1, keepdim=True)
        e = torch.where(took, torch.exp(value - top), zero)
        weights = torch.where(took, e / e.sum(1, keepdim=True), zero)
    elif c["score"] == "sigmoid":
        weights = torch.where(took, torch.exp(value), zero)
    else:
        top = logits.amax(1, keepdim=True)
        p = torch.where(mask, torch.exp(logits - top), torch.zeros_like(logits))
        p = torch.where(mask, p / p.sum(1, keepdim=True), p)
        weights = torch.where(took, p.gather(1, experts), zero)
    out = dict(weights=weights, experts=torch.where(took, experts, torch.full_like(experts, -1)).to(torch.int32))
    if c["backward"]:
        g = torch.where(took, s["dweights"], zero)
        if c["renormalize"]:
            d = weights * (g - (g * weights).sum(1, keepdim=True))
        elif c["score"] == "sigmoid":
            d = weights * g
        else:
            d = weights * g
        if c["score"] == "sigmoid":
            d = d / (1.0 + torch.exp(chosen))
        dlogits = torch.zeros_like(logits).scatter_add_(1, experts, torch.where(took, d, zero))
        if c["score"] == "softmax" and not c["renormalize"]:
            dlogits = dlogits - p * (g * weights).sum(1, keepdim=True)
        out["dlogits"] = dlogits.to(s["logits"].dtype)
    return out


def _gather(x, index):
    """Rows of x in 32 bits by index, zeros where it is negative."""
    got = x[index.clamp(min=0).long()].float()
    return torch.where((index >= 0)[..., None], got, torch.zeros((), device=x.device))


def _plain_dispatch(s, c):
    sizes, rows_of, source = _order(s["experts"], c["experts"])
    K = rows_of.shape[1]
    token = torch.where(source >= 0, source // K, source)
    out = dict(sizes=sizes, rows_of=rows_of, source=source, rows=_gather(s["x"], token).to(s["x"].dtype))
    if c["backward"]:
        out["dx"] = _gather(s["drows"], rows_of).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s, c):
    rows_of, source, weights, rows = s["rows_of"], s["source"], s["weights"], s["rows"]
    K = rows_of.shape[1]
    got = _gather(rows, rows_of)
    out = dict(out=(got * weights[..., None]).sum(1).to(rows.dtype))
    if c["backward"]:
        dout = s["dout"].float()
        token = torch.where(source >= 0, source // K, source)
        w = weights.reshape(-1)[source.clamp(min=0).long()]
        out["drows"] = (_gather(s["dout"], token) * w[:, None]).to(rows.dtype)
        out["dweights"] = (got * dout[:, None, :]).sum(2)
    return out


def _plain_quantize(s, c):
    return dict(values=_fp4(s["x"].float(), c["format"])[3].to(torch.bfloat16))


def _plain_product(s, c):
    K, D = s["rows_of"].shape[1], c["d"]
    token = torch.where(s["source"] >= 0, s["source"] // K, s["source"])
    values = _fp4(s["x"].float(), c["format"])[3]
    lhs = _gather(values, token)
    out = torch.zeros((lhs.shape[0], c["n"]), device="cuda", dtype=DTYPES[c["out"]])
    at = 0
    for g, size in enumerate(s["host_sizes"]):  # one product an expert, those without rows left out
        if size:
            w = _weight_values(s["codes"][g], s["scale"][g], None if s["row"] is None else s["row"][g], c["format"], D)
            out[at:at + size] = (lhs[at:at + size] @ w.T).to(out.dtype)
            at += size
    return dict(out=out)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    K = min(case.get("topk", 1), case.get("experts", 1))
    if op == "route":
        T, E, b = case["tokens"], case["experts"], BYTES[case["dtype"]]
        n = T * E * b + T * K * 8 + T
        if case["backward"]:
            n += T * E * b + T * K * 4
        return {"bytes": n, "flops": 4 * T * E}
    if op == "dispatch":
        T, D, b = case["tokens"], case["d"], BYTES[case["dtype"]]
        n = 3 * 4 * T * K + 4 * case["experts"] + T * D * b + T * K * D * b
        if case["backward"]:
            n += T * K * D * b + T * D * b
        return {"bytes": n, "flops": T * K * D if case["backward"] else 0}
    if op == "combine":
        T, D, b = case["tokens"], case["d"], BYTES[case["dtype"]]
        n = 8 * T * K + T * K * D * b + T * D * b
        if case["backward"]:
            n += T * D * b + T * K * D * b + 8 * T * K
        return {"bytes": n, "flops": (5 if case["backward"] else 2) * T * K * D}
    if op == "quantize":
        R, D, b = case["rows"], case["d"], BYTES[case["dtype"]]
        return {"bytes": R * D * (b + 2), "flops": 4 * R * D}
    T, E, D, N = case["tokens"], case["experts"], case["d"], case["n"]
    m = T * K
    used = E * (1.0 - (1.0 - K / E) ** T)  # experts that some token chooses, were all equally likely
    weights = used * N * (D / 2 + D / BLOCK[case["format"]])
    return {"bytes": T * D * 2 + weights + m * N * BYTES[case["out"]], "flops": 2 * m * N * D}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s, case)


def _exact_route(s, c):
    K, E = min(c["topk"], c["experts"]), c["experts"]
    logits, mask = s["logits"].double().cpu().numpy(), s["mask"].cpu().numpy()
    key = s["logits"].float()
    key = (key if s["bias"] is None else key + s["bias"]).cpu().numpy()  # the sum that selects is one of 32 bits
    T = logits.shape[0]
    logits[~mask], key[~mask] = -np.inf, -np.inf
    experts = np.argsort(-key, axis=1, kind="stable")[:, :K]
    took = np.take_along_axis(key, experts, 1) > -np.inf
    live = took.any(1)
    safe = np.where(mask[:, None], logits, 0.0)
    if c["score"] == "softmax":
        score = np.exp(safe - safe.max(1, keepdims=True))
        score /= score.sum(1, keepdims=True)
    else:
        score = 1.0 / (1.0 + np.exp(-safe))
    w = np.where(took, np.take_along_axis(score, experts, 1), 0.0)
    total = np.where(live, w.sum(1), 1.0)[:, None]
    weights = w / total if c["renormalize"] else w
    out = dict(weights=torch.from_numpy(weights), experts=None)
    if c["backward"]:
        g = np.where(took, s["dweights"].double().cpu().numpy(), 0.0)
        if c["renormalize"]:
            g = (g - (g * weights).sum(1, keepdims=True)) / total
        ds = np.zeros((T, E))
        np.put_along_axis(ds, experts, np.where(took, g, 0.0), 1)
        if c["score"] == "softmax":
            d = score * (ds - (ds * score).sum(1, keepdims=True))
        else:
            d = ds * score * (1.0 - score)
        out["dlogits"] = torch.from_numpy(np.where(mask[:, None], d, 0.0))
    return out


def _exact_dispatch(s, c):
    sizes, rows_of, source = (t.cpu() for t in _order(s["experts"], c["experts"]))
    T, K = rows_of.shape
    rows = torch.zeros((T * K, c["d"]), dtype=torch.float64, device="cuda")
    live = torch.nonzero(source >= 0).reshape(-1).cuda()
    rows[live] = s["x"].double()[torch.div(source.cuda()[live].long(), K, rounding_mode="floor")]
    out = dict(sizes=None, rows_of=None, source=None, rows=rows)
    if c["backward"]:
        dx = torch.zeros((T, c["d"]), dtype=torch.float64, device="cuda")
        for j in range(K):
            r = rows_of[:, j].cuda().long()
            t = torch.nonzero(r >= 0).reshape(-1)
            dx[t] += s["drows"][r[t]].double()
        out["dx"] = dx
    return out


def _exact_combine(s, c):
    rows_of, weights = s["rows_of"].long(), s["weights"].double()
    T, K = rows_of.shape
    total = torch.zeros((T, c["d"]), dtype=torch.float64, device="cuda")
    drows = torch.zeros((T * K, c["d"]), dtype=torch.float64, device="cuda")
    dweights = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for j in range(K):
        t = torch.nonzero(rows_of[:, j] >= 0).reshape(-1)
        r = rows_of[t, j]
        total[t] += weights[t, j, None] * s["rows"][r].double()
        if c["backward"]:
            drows[r] = weights[t, j, None] * s["dout"][t].double()
            dweights[t, j] = torch.einsum("td,td->t", s["dout"][t].double(), s["rows"][r].double())
    return dict(out=total, drows=drows, dweights=dweights) if c["backward"] else dict(out=total)


def _two_to(e):
    """2^e in 64 bits for whole e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_to(v, bits, least):
    """v >= 0 to `bits` bits after the first, spaced as for 2^least below it, ties to even."""
    e = torch.frexp(v)[1].to(torch.float64) - 1.0
    step = _two_to(torch.clamp(e, min=least) - bits)
    return torch.round(v / step) * step


def _exact_values(x, fmt):
    """The values that x [.., k] in 64 bits stands for in the format; all finite."""
    if fmt == "nvfp4":
        high = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(high > 0, high / 2688.0, torch.ones_like(high))))
        row = _two_to(e)
        row = torch.where(high > 2688.0 * row, row * 2, torch.where(high <= 1344.0 * row, row / 2, row))
        b = x.unflatten(-1, (-1, 16)) / row[..., None]
        s = _round_to(b.abs().amax(-1, keepdim=True) / 6.0, 3, -6.0)
    else:
        row = None
        b = x.unflatten(-1, (-1, 32))
        high = b.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(high > 0, high / 6.0, torch.ones_like(high))))
        s = _two_to(e)
        s = torch.where(high > 6.0 * s, s * 2, torch.where(high <= 3.0 * s, s / 2, s))
        s = torch.where(high > 0, s, torch.zeros_like(s))
    q = torch.where(s > 0, b.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b))
    q = _round_to(q, 1, 0.0).clamp(max=6.0)
    v = (torch.sign(b) * q * s).flatten(-2)
    return v if row is None else v * row


def _exact_quantize(s, c):
    return dict(values=_exact_values(s["x"].double(), c["format"]))


def _exact_product(s, c):
    D, fmt = c["d"], c["format"]
    K = s["rows_of"].shape[1]
    rows = _exact_values(s["x"].double(), fmt)
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.zeros((s["source"].numel(), c["n"]), dtype=torch.float64, device="cuda")
    ends = np.cumsum(s["host_sizes"])
    for g, (end, size) in enumerate(zip(ends, s["host_sizes"])):
        if size == 0:
            continue
        code = s["codes"][g]
        w = torch.empty((c["n"], D), dtype=torch.float64, device="cuda")
        for h in (0, 1):
            nib = (code >> (4 * h)) & 15
            w[:, h::2] = table[(nib & 7).long()] * torch.where(nib >= 8, -1.0, 1.0).double()
        at = torch.arange(D, device="cuda") // BLOCK[fmt]
        byte = s["scale"][g][at // 16, :, at % 16].T.double()
        if fmt == "nvfp4":
            e, f = torch.div(byte, 8, rounding_mode="floor"), byte % 8
            w *= torch.where(e > 0, (8 + f) * _two_to(e - 10), f * 2.0 ** -9) * s["row"][g].double()[:, None]
        else:
            w *= _two_to(byte - 127)
        token = torch.div(s["source"][end - size:end].long(), K, rounding_mode="floor")
        out[end - size:end] = rows[token] @ w.T
    return dict(out=out)
