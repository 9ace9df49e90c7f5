"""Plain 64-bit statements of the operators around the experts' products, in numpy: the router's
choice with its gradient, the order of tokens by expert with the ways there and back, and
microscaled 4-bit floating point."""

import numpy as np

U32 = 2.0 ** -24  # half the spacing of fp32 at 1
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ---------------------------------------------------------------- router
def choose(logits32, topk, select_bias32=None, mask=None):
    """experts [T, topk] (-1 where none): the largest fp32 sums logit + bias, ties by index."""
    key = logits32.astype(np.float32)
    if select_bias32 is not None:
        with np.errstate(invalid="ignore"):
            key = (key + select_bias32.astype(np.float32)).astype(np.float32)
    key = np.where(np.isnan(key), -np.inf, key)
    if mask is not None:
        key[~mask.astype(bool)] = -np.inf
    order = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    took = np.take_along_axis(key, order, 1) > -np.inf
    return np.where(took, order, -1)


def _scores(logits, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-logits))
        top = logits.max(axis=1, keepdims=True)
        e = np.exp(logits - np.where(np.isfinite(top), top, 0.0))
        return e / np.where(e.sum(1, keepdims=True) > 0, e.sum(1, keepdims=True), 1.0)


def weights_of(logits, experts, score, renormalize, scale):
    logits = np.where((experts >= 0).any(1, keepdims=True), logits, 0.0)
    s = _scores(logits, score)
    took = experts >= 0
    w = np.where(took, np.take_along_axis(s, np.maximum(experts, 0), 1), 0.0)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    return scale * w


def route_gradient(dweights, experts, logits, score, renormalize, scale):
    live = (experts >= 0).any(1, keepdims=True)
    logits = np.where(live, logits, 0.0)
    s = _scores(logits, score)
    took, at = experts >= 0, np.maximum(experts, 0)
    w = np.where(took, np.take_along_axis(s, at, 1), 0.0)
    g = np.where(took, scale * dweights, 0.0)
    if renormalize:
        total = np.where(live, w.sum(1, keepdims=True), 1.0)
        g = (g - (g * w).sum(1, keepdims=True) / total) / total
    ds = np.zeros_like(s)
    np.add.at(ds, (np.arange(len(s))[:, None], at), np.where(took, g, 0.0))
    d = s * (ds - (ds * s).sum(1, keepdims=True)) if score == "softmax" else ds * s * (1.0 - s)
    return np.where(live, d, 0.0)


# ---------------------------------------------------------------- order
def order_of(experts, num_experts):
    flat = experts.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < num_experts), flat, num_experts)
    slots = np.argsort(key, kind="stable")
    sizes = np.bincount(key, minlength=num_experts + 1)[:num_experts]
    n = int(sizes.sum())
    source = np.where(np.arange(flat.size) < n, slots, -1)
    rows = np.full(flat.size, -1)
    rows[slots[:n]] = np.arange(n)
    return sizes, rows.reshape(experts.shape), source


# ---------------------------------------------------------------- 4-bit
def _to_bits(v, bits, least):
    """v >= 0 rounded to `bits` bits after the first, ties to even, spaced as for 2^least below it."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, least) - bits)
    return np.rint(v / step) * step


def quantize(x, fmt):
    """(codes [.., k] 0..15, scale bytes [.., k / block], row scales or None) of x in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[:-1] + (-1, BLOCK[fmt]))
    bad = ~np.isfinite(b).all(-1)
    high = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    if fmt == "nvfp4":
        f, e = np.frexp(high.max(-1) / 2688.0)  # 2688 = 6 * 448
        e = np.where(np.ldexp(2688.0, e - 1) >= high.max(-1), e - 1, e)
        row = np.where(high.max(-1) > 0, np.ldexp(1.0, np.maximum(e, -126)), 1.0)
        s = _to_bits(high / row[..., None] / 6.0, 3, -6)
        _, se = np.frexp(s)
        ex = np.maximum(se - 1, -6)
        mant = (np.ldexp(s, 3 - ex)).astype(np.int64)  # 8..15, or 0..7 for subnormals
        byte = np.where(mant >= 8, ((ex + 7) << 3) + (mant - 8), mant)
        byte = np.where(bad, 0x7F, byte)
        whole = s * row[..., None]
    else:
        f, e = np.frexp(high / 6.0)
        e = np.where(np.ldexp(6.0, e - 1) >= high, e - 1, e)
        e = np.maximum(e, -127)
        s = np.where(high > 0, np.ldexp(1.0, e), 0.0)
        byte = np.where(bad, 255, np.where(high > 0, e + 127, 0))
        row, whole = None, s
    ok = (whole > 0) & ~bad
    q = np.abs(np.where(ok[..., None], b, 0.0)) / np.where(ok, whole, 1.0)[..., None]
    q = np.minimum(_to_bits(q, 1, 0), 6.0)
    code = np.searchsorted(E2M1, q) + 8 * np.where(bad[..., None], False, np.signbit(b))
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8), row


def scale_values(byte, fmt):
    byte = byte.astype(np.int64)
    if fmt == "mxfp4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    e, m = (byte >> 3) & 15, byte & 7
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(m.astype(np.float64), -9))
    return np.where((byte & 0x7F) == 0x7F, np.nan, v)


def values(codes, byte, row, fmt):
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    v = v.reshape(byte.shape + (BLOCK[fmt],)) * scale_values(byte, fmt)[..., None]
    v = v.reshape(codes.shape)
    return v if row is None else v * np.asarray(row, np.float64)[..., None]


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), axis=-1).reshape(packed.shape[:-1] + (-1,))


def to_windows(byte):
    """[.., rows, blocks] -> [.., windows, rows, 16], zeros past the last block."""
    nb = byte.shape[-1]
    w = -(-nb // 16)
    full = np.zeros(byte.shape[:-1] + (w * 16,), np.uint8)
    full[..., :nb] = byte
    return np.ascontiguousarray(np.moveaxis(full.reshape(byte.shape[:-1] + (w, 16)), -2, -3))


def from_windows(win, nb):
    full = np.moveaxis(win, -3, -2)
    return np.ascontiguousarray(full.reshape(full.shape[:-2] + (-1,))[..., :nb])
