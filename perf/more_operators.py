"""More operators of a mixture-of-experts layer: what is timed, and their plain forms.

  balance   the router's balance loss and z loss, the experts' loads, and the gradient of both losses
  gated     the gated activation between an expert's two products, with its gradient
  quantize  weights in 4-bit integers with a scale (and a zero point) for each group of k, and the values they stand for
  matvec    products of few tokens with the 4-bit weights of the experts that each chose, as a decoding step makes them

4-bit weights [.., n, k] are codes [.., n, k / 2] (the even k in the low nibble) with bf16 scales, and zero points in a byte,
by windows of 256 k: [.., ceil(k / 256), n, 256 / group].  Without zero points codes are two's complement, with them 0 to 15.
"""

import math

import torch

own = False

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
WINDOW = 256


def _gmm():
    import moe_grouped_matrix_gb300 as G

    return G


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a fine-tuning step's few tokens: all latency
        dict(name="balance_small", op="balance", tokens=192, experts=8, topk=2, sequences=1, dtype="bf16", score="softmax",
             dropped=0.0, backward=True),
        # the router of a training step, 8 of 128 experts for 4096 tokens
        dict(name="balance_train", op="balance", tokens=4096, experts=128, topk=8, sequences=1, dtype="bf16",
             score="softmax", dropped=0.0, backward=True),
        # a large batch of sequences, each balanced by itself, with sigmoid scores in f32 and slots dropped by capacity
        dict(name="balance_sequences", op="balance", tokens=16384, experts=250, topk=8, sequences=16, dtype="f32",
             score="sigmoid", dropped=0.05, backward=True),
        # a decoding step's rows between the two products
        dict(name="gated_decode", op="gated", rows=256, f=1024, dtype="bf16", act="silu", backward=False),
        # a training step of a 128-expert layer: 4096 tokens, 8 rows each
        dict(name="gated_train", op="gated", rows=32768, f=1024, dtype="bf16", act="silu", backward=True),
        # f32 rows of an odd width
        dict(name="gated_train_f32_odd", op="gated", rows=3001, f=2051, dtype="f32", act="gelu", backward=True),
        # the down projections of 8 experts packed for serving
        dict(name="quantize_experts", op="quantize", batch=8, n=4096, k=4096, group=128, zero_points=False, dtype="bf16"),
        # one matrix with a zero point for each 32 values
        dict(name="quantize_zero_points", op="quantize", batch=1, n=2048, k=4000, group=32, zero_points=True, dtype="f32"),
        # one token through the gate and up projections of 2 of 8 large experts, with the activation
        dict(name="matvec_up", op="matvec", tokens=1, experts=8, topk=2, n=28672, k=4096, group=128, zero_points=False,
             act="silu", per_slot=False, weighted=False, out="bf16"),
        # the same token's way back: the chosen experts' down projections, weighted and summed
        dict(name="matvec_down", op="matvec", tokens=1, experts=8, topk=2, n=4096, k=14336, group=128, zero_points=False,
             act="", per_slot=True, weighted=True, out="bf16"),
        # one token, 8 of 128 small experts: latency counts as much as bytes
        dict(name="matvec_small_experts", op="matvec", tokens=1, experts=128, topk=8, n=2048, k=2048, group=32,
             zero_points=False, act="silu", per_slot=False, weighted=False, out="bf16"),
        # a batch of 32 sequences' tokens, 4 of 64 experts each, weights with zero points
        dict(name="matvec_batch", op="matvec", tokens=32, experts=64, topk=4, n=2048, k=4096, group=64, zero_points=True,
             act="", per_slot=False, weighted=False, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "gated", "quantize", "matvec", "matvec"))
    if op == "balance":
        sequences = _log(rng, 1, 16)
        experts = _log(rng, 4, 256)
        return dict(op=op, tokens=sequences * _log(rng, 1, 1024), experts=experts, topk=rng.randint(1, min(8, experts)),
                    sequences=sequences, dtype=rng.choice(("bf16", "f32")), score=rng.choice(("softmax", "sigmoid")),
                    dropped=rng.choice((0.0, 0.1)), backward=rng.random() < 0.7)
    if op == "gated":
        return dict(op=op, rows=_log(rng, 1, 16384), f=_log(rng, 16, 2048), dtype=rng.choice(("bf16", "f32")),
                    act=rng.choice(("silu", "gelu")), backward=rng.random() < 0.5)
    group = rng.choice((32, 64, 128))
    if op == "quantize":
        return dict(op=op, batch=_log(rng, 1, 8), n=_log(rng, 1, 2048), k=group * _log(rng, 1, 4096 // group), group=group,
                    zero_points=rng.random() < 0.5, dtype=rng.choice(("bf16", "f32")))
    experts = _log(rng, 1, 32)
    tokens = _log(rng, 1, 32)
    weighted = rng.random() < 0.4
    act = "" if weighted else rng.choice(("", "silu", "gelu"))
    return dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(8, experts, 128 // tokens)),
                n=16 * _log(rng, 4, 128), k=group * _log(rng, 1, 4096 // group), group=group,
                zero_points=rng.random() < 0.5, act=act, per_slot=weighted or rng.random() < 0.2, weighted=weighted,
                out=rng.choice(("bf16", "bf16", "f32")))


# ---------------------------------------------------------------- inputs
def _choice(score, topk):
    return torch.sort(score, dim=1, descending=True, stable=True)[1][:, :topk].to(torch.int32).contiguous()


def _groups(x, group, zero_points):
    """x [.., k] in 32 bits as (codes held in bytes, scales in bf16, zero points or None), by groups of k."""
    g = x.unflatten(-1, (-1, group))
    if zero_points:
        low, high = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
        span, steps, least, most = high - low, 15.0, 0.0, 15.0
    else:
        span, steps, least, most = g.abs().amax(-1), 7.0, -8.0, 7.0
    fine = torch.isfinite(span)
    scale = (span / torch.full_like(span, steps)).to(torch.bfloat16)
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    s = scale.float()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    q = torch.round(g / safe[..., None])
    zero = None
    if zero_points:
        zero = torch.where(s > 0, torch.round(-low / safe).clamp(0.0, 15.0), torch.zeros_like(s))
        q = q + zero[..., None]
    q = torch.where((s > 0)[..., None], q.clamp(least, most), torch.zeros_like(q))
    return q.flatten(-2).to(torch.int8), scale, zero if zero is None else zero.to(torch.uint8)


def _windows(t, group):
    """Values of groups [.., n, k / group] by windows of k, zeros past the end."""
    each = WINDOW // group
    w = -(-t.shape[-1] // each)
    full = torch.zeros(t.shape[:-1] + (w * each,), dtype=t.dtype, device=t.device)
    full[..., : t.shape[-1]] = t
    return full.unflatten(-1, (w, each)).transpose(-3, -2).contiguous()


def _values(codes, scale, zero, group, k):
    """The values, in 32 bits, that packed weights [.., n, k] stand for."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    s = scale.transpose(-3, -2).flatten(-2)[..., : k // group].float()
    if zero is None:
        q = torch.where(q > 7, q - 16, q).unflatten(-1, (-1, group))
    else:
        q = q.unflatten(-1, (-1, group)) - zero.transpose(-3, -2).flatten(-2)[..., : k // group].float()[..., None]
    return (q * s[..., None]).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std, dtype=torch.float32):
        return (std * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    op, s = case["op"], dict(case=case)
    if op == "balance":
        T, E, K = case["tokens"], case["experts"], case["topk"]
        dtype = DTYPES[case["dtype"]]
        logits = (normal((1, E), 0.8) + normal((T, E), 1.5)).to(dtype)  # some experts are liked more than others
        if E > K:
            logits[:, seed % E] = -math.inf  # an expert that is switched off
        experts = _choice(logits.float(), K)
        mask = torch.rand(T, generator=gen, device="cuda") > 0.03
        mask[0] = True
        if case["sequences"] > 2:  # a sequence that is padding from end to end
            L = T // case["sequences"]
            mask[L: 2 * L] = False
        logits[~mask] = math.nan  # padding tokens: what is there does not count
        gone = ~mask[:, None]
        if case["dropped"]:
            gone = gone | (torch.rand((T, K), generator=gen, device="cuda") < case["dropped"])
        s.update(logits=logits, mask=mask, experts=torch.where(gone, torch.full_like(experts, -1), experts),
                 dlosses=torch.rand(2, generator=gen, device="cuda") * 0.01 + 0.01 if case["backward"] else None)
    elif op == "gated":
        m, f, dtype = case["rows"], case["f"], DTYPES[case["dtype"]]
        h = normal((m, 2 * f), 1.5, dtype)
        if m > 8:
            h[-(m // 8):] = 0  # rows past the experts' groups
        s.update(h=h, dout=normal((m, f), 0.01, dtype) if case["backward"] else None)
    elif op == "quantize":
        x = normal((case["batch"], case["n"], case["k"]), 0.02)
        x[..., seed % case["k"]] *= 20.0  # a channel that stands out
        x[0, 0, : case["group"]] = 0.0
        s.update(x=x.to(DTYPES[case["dtype"]]))
    else:
        T, E, K, n, k, group = (case[name] for name in ("tokens", "experts", "topk", "n", "k", "group"))
        each = WINDOW // group
        windows = -(-k // WINDOW)
        codes = torch.empty((E, n, k // 2), dtype=torch.uint8, device="cuda")
        scale = torch.empty((E, windows, n, each), dtype=torch.bfloat16, device="cuda")
        zero = torch.empty((E, windows, n, each), dtype=torch.uint8, device="cuda") if case["zero_points"] else None
        for e in range(E):
            q, sc, z = _groups(normal((n, k), 0.02), group, case["zero_points"])
            q = q.to(torch.uint8) & 15
            codes[e] = q[:, 0::2] | (q[:, 1::2] << 4)
            scale[e] = _windows(sc, group)
            if zero is not None:
                zero[e] = _windows(z, group)
        experts = _choice(normal((1, E), 0.6) + normal((T, E), 1.0), K)
        s.update(codes=codes, scale=scale, zero=zero, experts=experts, host_experts=experts.tolist(),
                 x=normal((T, K, k) if case["per_slot"] else (T, k), 1.0, torch.bfloat16),
                 weights=torch.softmax(normal((T, K), 1.0), dim=1) if case["weighted"] else None)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](s, s["case"])


def _own_balance(s, c):
    G = _gmm()
    b = G.balance_loss(s["logits"], s["experts"], score=c["score"], token_mask=s["mask"], sequences=c["sequences"])
    out = dict(losses=b.losses, counts=b.counts, tokens=b.tokens)
    if c["backward"]:
        out["dlogits"] = G.balance_loss_backward(s["dlosses"], b, s["logits"], score=c["score"], token_mask=s["mask"])
    return out


def _own_gated(s, c):
    G = _gmm()
    out = dict(out=G.gated_act(s["h"], c["act"]))
    if c["backward"]:
        out["dh"] = G.gated_act_backward(s["dout"], s["h"], c["act"])
    return out


def _own_quantize(s, c):
    G = _gmm()
    return dict(values=G.dequantize_int4(G.quantize_int4(s["x"], c["group"], zero_points=c["zero_points"])))


def _own_matvec(s, c):
    G = _gmm()
    w = G.Int4Tensor(s["codes"], s["scale"], s["zero"], c["group"])
    return dict(out=G.matvec_int4(s["x"], w, s["experts"], weights=s["weights"], act=c["act"] or None,
                                  out_dtype=DTYPES[c["out"]]))


def _plain_balance(s, c):
    S, E, score = c["sequences"], c["experts"], c["score"]
    live = s["mask"]
    zero = torch.zeros((), device="cuda")
    l = torch.where(live[:, None], s["logits"].float(), zero)
    index = torch.where(live[:, None] & (s["experts"] >= 0), s["experts"].long(), E)
    T = l.shape[0]
    at = torch.arange(T, device="cuda")[:, None] // (T // S)
    counts = torch.zeros(S * (E + 1), dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, (at * (E + 1) + index).reshape(-1), torch.ones(index.numel(), dtype=torch.int32, device="cuda"))
    counts = counts.reshape(S, E + 1)[:, :E].contiguous()
    tokens = live.sum().to(torch.int32).reshape(1)
    N = tokens.float().clamp(min=1.0)
    share = counts.float() / counts.sum(1, keepdim=True).clamp(min=1).float()
    share = share.repeat_interleave(T // S, dim=0)

    def softmax(v):
        high = v.amax(1, keepdim=True)
        e = torch.exp(v - high)
        total = e.sum(1, keepdim=True)
        return e / total, high + torch.log(total)

    q, lse = softmax(l)
    if score == "sigmoid":
        p, _ = softmax(torch.clamp(l, max=0.0) - torch.log1p(torch.exp(-l.abs())))
    else:
        p = q
    mean = (share * p).sum(1, keepdim=True)  # of a token's experts' shares
    of = live[:, None]
    losses = torch.stack((E * torch.where(of, mean, zero).sum() / N[0], torch.where(of, lse * lse, zero).sum() / N[0]))
    out = dict(losses=losses, counts=counts, tokens=tokens)
    if c["backward"]:
        d = (s["dlosses"][0] * E / N) * p * (share - mean)
        if score == "sigmoid":
            d = d / (1.0 + torch.exp(l))
        d = d + (s["dlosses"][1] * 2.0 / N) * lse * q
        out["dlogits"] = torch.where(of, d, zero).to(s["logits"].dtype)
    return out


def _plain_gated(s, c):
    f = c["f"]
    g, u = s["h"][:, :f].float(), s["h"][:, f:].float()
    if c["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        a, da = g * sig, sig * (1.0 + g * (1.0 - sig))
    else:
        inner = 0.7978845608028654 * (g + 0.044715 * g * g * g)
        sig = 1.0 / (1.0 + torch.exp(-2.0 * inner))  # (1 + tanh(inner)) / 2
        a = g * sig
        da = sig + g * 2.0 * sig * (1.0 - sig) * 0.7978845608028654 * (1.0 + 3.0 * 0.044715 * g * g)
    out = dict(out=(a * u).to(s["h"].dtype))
    if c["backward"]:
        d = s["dout"].float()
        out["dh"] = torch.cat((d * u * da, d * a), dim=1).to(s["h"].dtype)
    return out


def _plain_quantize(s, c):
    q, scale, zero = _groups(s["x"].float(), c["group"], c["zero_points"])
    v = q.float().unflatten(-1, (-1, c["group"]))
    if zero is not None:
        v = v - zero.float()[..., None]
    return dict(values=(v * scale.float()[..., None]).flatten(-2).to(torch.bfloat16))


def _act(h, act):
    f = h.shape[-1] // 2
    g, u = h[..., :f], h[..., f:]
    if act == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    return g / (1.0 + torch.exp(-1.5957691216057308 * (g + 0.044715 * g * g * g))) * u


def _plain_matvec(s, c):
    T, K, n, k = c["tokens"], c["topk"], c["n"], c["k"]
    x = s["x"].float()
    slots = {}
    for t, row in enumerate(s["host_experts"]):
        for j, e in enumerate(row):
            slots.setdefault(e, []).append((t, j))
    h = torch.zeros((T, K, n), device="cuda")
    for e, at in slots.items():  # one product an expert, those that no token chose left out
        w = _values(s["codes"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e], c["group"], k)
        t, j = (torch.tensor(v, device="cuda") for v in zip(*at))
        h[t, j] = (x[t, j] if c["per_slot"] else x[t]) @ w.T
    if c["act"]:
        h = _act(h, c["act"])
    if c["weighted"]:
        h = (h * s["weights"][..., None]).sum(1)
    return dict(out=h.to(DTYPES[c["out"]]))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "balance":
        T, E, b = case["tokens"], case["experts"], BYTES[case["dtype"]]
        n = T * E * b + 4 * T * case["topk"] + T + 4 * case["sequences"] * E
        return {"bytes": n + (T * E * b if case["backward"] else 0), "flops": (16 if case["backward"] else 6) * T * E}
    if op == "gated":
        n = case["rows"] * case["f"]
        return {"bytes": (6 if case["backward"] else 3) * n * BYTES[case["dtype"]],
                "flops": (20 if case["backward"] else 6) * n}
    if op == "quantize":
        n = case["batch"] * case["n"] * case["k"]
        return {"bytes": n * (BYTES[case["dtype"]] + 2), "flops": 4 * n}
    T, E, K, n, k = (case[name] for name in ("tokens", "experts", "topk", "n", "k"))
    used = E * (1.0 - (1.0 - K / E) ** T)  # experts that some token chooses, were all equally likely
    weights = used * n * (k / 2 + (3 if case["zero_points"] else 2) * (k // case["group"]))
    rows = T * (1 if case["weighted"] else K) * (n // 2 if case["act"] else n)
    return {"bytes": weights + 2 * T * (K if case["per_slot"] else 1) * k + rows * BYTES[case["out"]],
            "flops": 2 * T * K * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s, case)


def _exact_balance(s, c):
    S, E, T = c["sequences"], c["experts"], c["tokens"]
    L = T // S
    live = torch.nonzero(s["mask"]).reshape(-1)
    N = live.numel()
    l = s["logits"][live].double()
    chosen = s["experts"][live]
    seq = torch.div(live, L, rounding_mode="floor")
    share = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    for j in range(c["topk"]):
        kept = chosen[:, j] >= 0
        share.index_put_((seq[kept], chosen[kept, j].long()), torch.ones((), dtype=torch.float64, device="cuda"),
                         accumulate=True)
    share = share / share.sum(1, keepdim=True).clamp(min=1.0)
    share = share[seq]
    lse = torch.logsumexp(l, dim=1, keepdim=True)
    soft = torch.exp(l - lse)
    if c["score"] == "sigmoid":
        sig = 1.0 / (1.0 + torch.exp(-l))
        p = sig / sig.sum(1, keepdim=True)
    else:
        sig, p = None, soft
    mean = (share * p).sum(1, keepdim=True)
    out = dict(losses=torch.stack((E * mean.sum() / N, (lse ** 2).sum() / N)), counts=None, tokens=None)
    if c["backward"]:
        d0, d1 = s["dlosses"].double()
        d = d0 * E / N * p * (share - mean)
        if sig is not None:
            d = d * (1.0 - sig)
        full = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        full[live] = d + d1 * 2.0 / N * lse * soft
        out["dlogits"] = full
    return out


def _exact_gated(s, c):
    g, u = s["h"].double().chunk(2, dim=1)
    if c["act"] == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * (1.0 - sig)
    else:
        root = math.sqrt(2.0 / math.pi)
        th = torch.tanh(root * (g + 0.044715 * g ** 3))
        a = 0.5 * g * (1.0 + th)
        da = 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * root * (1.0 + 3 * 0.044715 * g ** 2)
    out = dict(out=a * u)
    if c["backward"]:
        d = s["dout"].double()
        out["dh"] = torch.cat((d * u * da, d * a), dim=1)
    return out


def _exact_quantize(s, c):
    x = s["x"].double().unflatten(-1, (-1, c["group"]))
    if c["zero_points"]:
        low, high = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
        span = (high - low).float().double()  # the spread and its quotient are ones of 32 bits
        scale = (span / 15).float().to(torch.bfloat16).double()
        safe = torch.where(scale > 0, scale, 1.0)
        zero = torch.round(-low / safe).clamp(0, 15)
        v = (torch.round(x / safe) + zero).clamp(0, 15) - zero
    else:
        scale = (x.abs().amax(-1, keepdim=True) / 7).float().to(torch.bfloat16).double()
        v = torch.round(x / torch.where(scale > 0, scale, 1.0)).clamp(-8, 7)
    return dict(values=(v * scale).flatten(-2))


def _exact_matvec(s, c):
    T, K, n, k, group = (c[name] for name in ("tokens", "topk", "n", "k", "group"))
    each = WINDOW // group
    h = torch.zeros((T, K, n), dtype=torch.float64, device="cuda")
    at = torch.arange(k // group, device="cuda")
    for e in sorted({e for row in s["host_experts"] for e in row}):
        code = s["codes"][e].to(torch.int16)
        w = torch.empty((n, k), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (code % 16).double(), torch.div(code, 16, rounding_mode="floor").double()
        where = torch.div(at, each, rounding_mode="floor"), at % each
        scale = s["scale"][e][where[0], :, where[1]].T.double().repeat_interleave(group, dim=1)
        if s["zero"] is None:
            w = (w + 8) % 16 - 8
        else:
            w -= s["zero"][e][where[0], :, where[1]].T.double().repeat_interleave(group, dim=1)
        w *= scale
        for t, row in enumerate(s["host_experts"]):
            for j in range(K):
                if row[j] == e:
                    h[t, j] = w @ (s["x"][t, j] if c["per_slot"] else s["x"][t]).double()
    if c["act"]:
        g, u = h.chunk(2, dim=2)
        if c["act"] == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))) * u
    if c["weighted"]:
        h = (h * s["weights"].double()[..., None]).sum(1)
    return dict(out=h)
