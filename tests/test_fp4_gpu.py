"""quantize_fp4(), dequantize_fp4() and gmm_fp4() against the 64-bit statement.

Quantisation and its inverse are exact: codes, scale bytes and row scales are compared bit for bit.
The product's terms are exact; the tensor cores add them in fp32.  With at most k / 16 additions of
block sums, each off by no more than 2^-21 of the running magnitude (two bits of alignment loss on
top of a unit), the bound is (k / 16 + 8) * 2^-21 of the sum of magnitudes, and half a unit of the
output's format."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G
import moe_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMATS = ["nvfp4", "mxfp4"]
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -23}


def as64(t):
    return t.detach().cpu().double().numpy()


def check_quantized(q, x64, fmt):
    """The Fp4Tensor's bits against those of x64 [.., rows, k]."""
    codes, byte, row = R.quantize(x64, fmt)
    np.testing.assert_array_equal(q.block_scale.cpu().numpy(), R.to_windows(byte))
    if row is None:
        assert q.row_scale is None
    else:
        np.testing.assert_array_equal(as64(q.row_scale), row)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), R.pack(codes))
    return R.values(codes, byte, row, fmt)


def spread(rows, k, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, k), generator=gen) * torch.exp(2 * torch.randn((rows, 1), generator=gen))
    x *= torch.exp(2 * torch.randn((1, k), generator=gen))
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (5, 224), (70, 256), (9, 288), (33, 512), (130, 1024), (4, 1056),
                                    (65, 4096), (3, 4128), (2, 20000)])
def test_quantize(rows, k, dtype, fmt):
    x = spread(rows, k, dtype, rows + k)
    x[rows // 2, : k // 2] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = -0.0
    q = G.quantize_fp4(x.to(DEV), fmt)
    v = check_quantized(q, as64(x), fmt)
    for out in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(as64(G.dequantize_fp4(q, out)), v)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_half_way_point(fmt):
    """Values half way between two codes for every significand a scale can have, and one fp32 step to
    each side of them: the nearest code, the even one on the point itself."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for mant in range(8, 16):
        s = np.float32(mant / 8.0) if fmt == "nvfp4" else np.float32(1.0)
        for to in (-np.inf, None, np.inf):
            v = (ties * s).astype(np.float32)
            v = v if to is None else np.nextafter(v, np.float32(to))
            block = np.concatenate([[6 * s], v, -v, [0.0]]).astype(np.float32)
            rows.append(np.concatenate([np.full(16, 6 * 448, np.float32), block] if fmt == "nvfp4" else [block, block]))
    x = torch.from_numpy(np.stack(rows))
    check_quantized(G.quantize_fp4(x.to(DEV), fmt), as64(x), fmt)


def test_every_half_way_scale():
    """Block maxima at 6 times the points half way between two e4m3 values, and a step to each side."""
    steps = np.concatenate([np.arange(16) * 2.0 ** -9] + [(8 + np.arange(8)) * 2.0 ** e for e in range(-8, 6)])
    steps = np.unique(steps[steps <= 448])
    mid = (steps[1:] + steps[:-1]) / 2
    a = (6 * mid).astype(np.float32)
    a = np.concatenate([a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(np.inf))])
    x = np.zeros((1, 16 * (len(a) + 1 + (len(a) + 1) % 2)), np.float32)
    x[0, 0] = 6 * 448
    x[0, 16:16 * (len(a) + 1):16] = a
    x = torch.from_numpy(x)
    check_quantized(G.quantize_fp4(x.to(DEV), "nvfp4"), as64(x), "nvfp4")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_ends_of_the_range(fmt, dtype):
    info = torch.finfo(dtype)
    x = torch.zeros((8, 64), dtype=dtype)
    x[0] = info.max
    x[1] = -info.max
    x[2] = info.tiny
    x[3] = info.smallest_normal * 2.0 ** -6
    x[4, :16], x[4, 16:] = info.max, info.tiny
    x[5, 3] = 2.0 ** -126
    x[6, 40] = 1.0
    x[7] = 6 * 448 * 2.0 ** 20
    check_quantized(G.quantize_fp4(x.to(DEV), fmt), as64(x), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [256, 4096])
def test_what_is_not_finite_spoils_its_block_alone(fmt, dtype, k):
    x = spread(6, k, dtype, 4)
    x[0, 5], x[1, 40], x[2, 64:] = float("nan"), float("inf"), -float("inf")
    x[3] = float("nan")
    q = G.quantize_fp4(x.to(DEV), fmt)
    v = check_quantized(q, as64(x), fmt)
    got = as64(G.dequantize_fp4(q, torch.float32))
    np.testing.assert_array_equal(got, v)
    block = R.BLOCK[fmt]
    assert np.isnan(got[0]).sum() == block and np.isnan(got[1]).sum() == block and np.isnan(got[3]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_batches_pitches_and_odd_addresses(fmt):
    x = spread(3 * 40, 320, torch.bfloat16, 6).to(DEV)
    q = G.quantize_fp4(x.view(3, 40, 320), fmt)
    check_quantized(q, as64(x).reshape(3, 40, 320), fmt)
    v = G.dequantize_fp4(q)
    for b in range(3):
        one = G.quantize_fp4(x.view(3, 40, 320)[b], fmt)
        assert torch.equal(one.codes, q.codes[b]) and torch.equal(one.block_scale, q.block_scale[b])
        assert torch.equal(G.dequantize_fp4(one), v[b])
    for dtype in (torch.bfloat16, torch.float32):
        wide = x.to(dtype)
        for lo in (0, 1, 8):
            view = wide[:, lo:lo + 288]
            check_quantized(G.quantize_fp4(view, fmt), as64(view), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,topk,k,dropped", [(1, 4, 256, 0.0), (40, 3, 288, 0.3), (64, 4, 4096, 0.0),
                                                   (7, 32, 2048, 0.5), (5, 2, 96, 1.0)])
def test_rows_in_expert_order(tokens, topk, k, dropped, fmt):
    gen = torch.Generator().manual_seed(1)
    e = torch.randint(0, 9, (tokens, topk), generator=gen).to(torch.int32)
    e[torch.rand((tokens, topk), generator=gen) < dropped] = -1
    order = G.sort_by_expert(e.to(DEV), 9)
    x = spread(tokens, k, torch.bfloat16, 8).to(DEV)
    q = G.quantize_fp4(x, fmt, order=order)
    want = G.quantize_fp4(G.dispatch(x, order), fmt)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.block_scale, want.block_scale)
    assert fmt == "mxfp4" or torch.equal(q.row_scale, want.row_scale)


# ---------------------------------------------------------------- product
def operand(shape, fmt, seed, std=1.0):
    """An Fp4Tensor on the GPU of normal values, and its values in 64 bits."""
    gen = torch.Generator().manual_seed(seed)
    x = (std * torch.randn(shape, generator=gen)).numpy()
    codes, byte, row = R.quantize(x, fmt)
    q = G.Fp4Tensor(torch.from_numpy(R.pack(codes)).to(DEV), torch.from_numpy(R.to_windows(byte)).to(DEV),
                    None if row is None else torch.from_numpy(row).float().to(DEV), fmt)
    return q, R.values(codes, byte, row, fmt)


def check_product(out, a, w, sizes, offset, bias, k):
    m, n = out.shape
    ref, mag = np.zeros((m, n)), np.zeros((m, n))
    ends = np.minimum(np.cumsum(np.maximum(sizes, 0)), m)
    starts = np.concatenate([[0], ends[:-1]])
    for l in range(w.shape[0]):
        lo, hi = starts[offset + l], ends[offset + l]
        b = 0.0 if bias is None else bias[l]
        ref[lo:hi] = a[lo:hi] @ w[l].T + b
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(w[l]).T + np.abs(b)
    err = np.abs(as64(out) - ref)
    assert (err <= (k / 16 + 8) * 2.0 ** -21 * mag + UNIT[out.dtype] * np.abs(ref)).all(), (err / (mag + 1e-30)).max()


PRODUCTS = [
    # sizes, rows past the groups, k, n
    ([4], 0, 256, 128),
    ([1], 0, 32, 8),
    ([0, 1, 0, 3], 0, 64, 136),
    ([16, 16], 0, 512, 256),
    ([5, 0, 130, 17], 9, 320, 264),
    ([225, 1, 500], 3, 768, 200),
    ([33, 224, 448], 0, 1024, 384),
    ([0, 0, 0], 20, 128, 64),
    ([3, 1, 4, 1, 5, 9, 2, 6] * 8, 0, 288, 96),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_product(case, out_dtype, fmt):
    sizes, rest, k, n = PRODUCTS[case]
    m = sum(sizes) + rest
    lhs, a = operand((m, k), fmt, 1)
    rhs, w = operand((len(sizes), n, k), fmt, 2, 0.1)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    bias = None
    if case % 2:
        bias = torch.randn((len(sizes), 1, n), generator=torch.Generator().manual_seed(3))
        bias = bias.to(torch.bfloat16 if case % 4 == 1 else torch.float32).to(DEV)
    out = G.gmm_fp4(lhs, rhs, gs, rhs_bias=bias, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert G.read_device_errors() == 0
    check_product(out, a, w, sizes, 0, None if bias is None else as64(bias), k)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name,groups,mean,k,n", [("few rows", 64, 4, 4096, 1024), ("some rows", 32, 12, 2080, 2048),
                                                  ("many rows", 8, 700, 4096, 4096), ("ragged", 128, 60, 1056, 1032)])
def test_long_runs_of_tiles(name, groups, mean, k, n, out_dtype, fmt):
    """Several tiles for every SM and many times the pipeline's stages for each, several times over."""
    rng = np.random.default_rng(groups)
    sizes = rng.poisson(mean * rng.exponential(1.0, groups))
    m = int(sizes.sum()) + 3
    x = torch.randn((m, k), device=DEV).to(torch.bfloat16)
    wv = (0.1 * torch.randn((groups, n, k), device=DEV)).to(torch.bfloat16)
    lhs, rhs = G.quantize_fp4(x, fmt), G.quantize_fp4(wv, fmt)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    first = G.gmm_fp4(lhs, rhs, gs, out_dtype=out_dtype)
    for _ in range(4):
        assert torch.equal(G.gmm_fp4(lhs, rhs, gs, out_dtype=out_dtype), first)
    assert G.read_device_errors() == 0
    a, w = G.dequantize_fp4(lhs, torch.float32), G.dequantize_fp4(rhs, torch.float32)
    at = 0
    for g, size in enumerate(sizes.tolist()):
        a64, w64, got = a[at:at + size].double(), w[g].double(), first[at:at + size].double()
        ref, mag = a64 @ w64.T, a64.abs() @ w64.abs().T
        assert ((got - ref).abs() <= (k / 16 + 8) * 2.0 ** -21 * mag + UNIT[out_dtype] * ref.abs()).all(), g
        at += size
    assert first[at:].abs().max() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_and_scale(fmt):
    """Each e2m1 code against each, and each finite scale byte, one block at a time (sums of one term)."""
    k = R.BLOCK[fmt] * 16
    codes = np.zeros((32, k), np.uint8)
    codes[:16, 0] = np.arange(16)
    codes[16:, k // 2 + 1] = np.arange(16)
    byte = np.full((32, 16), 0x38 if fmt == "nvfp4" else 127, np.uint8)
    wbytes = (np.arange(127) if fmt == "nvfp4" else np.arange(40, 214)).astype(np.uint8)
    n = 176
    wcodes = np.full((1, n, k), 2, np.uint8)
    wbyte = np.resize(wbytes, n)[None, :, None].repeat(16, 2)
    ones = (lambda s: torch.ones(s, device=DEV)) if fmt == "nvfp4" else (lambda s: None)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    lhs = G.Fp4Tensor(dev(R.pack(codes)), dev(R.to_windows(byte)), ones((32,)), fmt)
    rhs = G.Fp4Tensor(dev(R.pack(wcodes)), dev(R.to_windows(wbyte)), ones((1, n)), fmt)
    out = G.gmm_fp4(lhs, rhs, torch.tensor([32], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    want = R.values(codes, byte, None, fmt) @ R.values(wcodes, wbyte, None, fmt)[0].T
    np.testing.assert_array_equal(as64(out), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_each_block_meets_its_own_scales(fmt):
    """One code a block and scales that are powers of two of the block, the row and the column: a sum
    that any misplaced scale would change."""
    k, m, n = 1024, 250, 264
    block = R.BLOCK[fmt]
    nb = k // block
    rng = np.random.default_rng(0)
    codes = np.zeros((m, k), np.uint8)
    codes[:, ::block] = 2
    wcodes = np.zeros((1, n, k), np.uint8)
    wcodes[:, :, ::block] = 2
    lo, mid = (0x20, 8) if fmt == "nvfp4" else (120, 1)
    byte = (lo + mid * rng.integers(0, 6, (m, nb))).astype(np.uint8)
    wbyte = (lo + mid * rng.integers(0, 6, (1, n, nb))).astype(np.uint8)
    one = (lambda s: torch.ones(s, device=DEV)) if fmt == "nvfp4" else (lambda s: None)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    lhs = G.Fp4Tensor(dev(R.pack(codes)), dev(R.to_windows(byte)), one((m,)), fmt)
    rhs = G.Fp4Tensor(dev(R.pack(wcodes)), dev(R.to_windows(wbyte)), one((1, n)), fmt)
    out = G.gmm_fp4(lhs, rhs, torch.tensor([m], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    want = R.values(codes, byte, None, fmt) @ R.values(wcodes, wbyte, None, fmt)[0].T
    np.testing.assert_array_equal(as64(out), want)  # sums of at most 64 terms within 10 binades: exact


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_slice_of_the_groups(fmt):
    sizes, k, n = [7, 40, 0, 130, 21], 256, 128
    m = sum(sizes) + 5
    lhs, a = operand((m, k), fmt, 4)
    rhs, w = operand((5, n, k), fmt, 5)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    for first, count in ((0, 2), (1, 3), (4, 1)):
        part = G.Fp4Tensor(rhs.codes[first:first + count].contiguous(), rhs.block_scale[first:first + count].contiguous(),
                           None if rhs.row_scale is None else rhs.row_scale[first:first + count].contiguous(), fmt)
        out = torch.full((m, n), float("nan"), device=DEV)
        G.gmm_fp4(lhs, part, gs, group_offset=first, out=out)
        check_product(out, a, w[first:first + count], np.array(sizes), first, None, k)


def test_bad_group_sizes_are_reported():
    lhs, a = operand((20, 64), "nvfp4", 6)
    rhs, w = operand((2, 16, 64), "nvfp4", 7)
    for sizes, flag in (([-3, 20], G.DEVERR_NEGATIVE_GROUP_SIZE), ([15, 15], G.DEVERR_GROUP_SIZES_EXCEED_M)):
        G.read_device_errors()
        out = G.gmm_fp4(lhs, rhs, torch.tensor(sizes, dtype=torch.int32, device=DEV), out_dtype=torch.float32)
        assert G.read_device_errors() == flag
        check_product(out, a, w, np.array(sizes), 0, None, 64)


def test_a_nan_block_spoils_its_row_alone():
    k, n = 512, 128
    for fmt in FORMATS:
        x = torch.randn((40, k), generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
        x[11, 300] = float("inf")
        lhs = G.quantize_fp4(x.to(DEV), fmt)
        rhs, w = operand((1, n, k), fmt, 10)
        out = G.gmm_fp4(lhs, rhs, torch.tensor([40], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
        bad = torch.isnan(out)
        assert bad[11].all() and bad.sum() == n


def test_offsets_past_32_bits():
    m, k, n = 140000, 256, 16384  # 2.3e9 outputs
    x = torch.randn((m, k), device=DEV).to(torch.bfloat16)
    wv = torch.randn((2, n, k), device=DEV).to(torch.bfloat16)
    lhs, rhs = G.quantize_fp4(x, "nvfp4"), G.quantize_fp4(wv, "nvfp4")
    out = G.gmm_fp4(lhs, rhs, torch.tensor([m - 5000, 5000], dtype=torch.int32, device=DEV))
    a, w = G.dequantize_fp4(lhs, torch.float32).double(), G.dequantize_fp4(rhs, torch.float32).double()
    for rows, g in ((slice(0, 300), 0), (slice(m - 5300, m - 5000), 0), (slice(m - 300, m), 1)):
        ref, mag = a[rows] @ w[g].T, a[rows].abs() @ w[g].abs().T
        assert ((out[rows].double() - ref).abs() <= 24 * 2.0 ** -21 * mag + 2.0 ** -8 * ref.abs()).all()


def test_another_stream_and_a_graph():
    lhs, a = operand((100, 512), "mxfp4", 11)
    rhs, w = operand((4, 256, 512), "mxfp4", 12)
    gs = torch.tensor([40, 0, 50, 10], dtype=torch.int32, device=DEV)
    want = G.gmm_fp4(lhs, rhs, gs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = G.gmm_fp4(lhs, rhs, gs)
    s.synchronize()
    assert torch.equal(got, want)
    G.workspace_for(torch.device(DEV))
    graph = torch.cuda.CUDAGraph()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(graph):
        got = G.gmm_fp4(lhs, rhs, gs, workspace=ws)
    gs.copy_(torch.tensor([0, 100, 0, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, G.gmm_fp4(lhs, rhs, gs)) and not torch.equal(got, want)


def test_none_at_all():
    rhs, _ = operand((2, 16, 64), "nvfp4", 13)
    q = G.quantize_fp4(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV))
    assert G.dequantize_fp4(q).shape == (0, 64)
    assert G.gmm_fp4(q, rhs, torch.zeros(2, dtype=torch.int32, device=DEV)).shape == (0, 16)


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="multiple of 32"):
        G.quantize_fp4(x[:, :48].contiguous())
    with pytest.raises(ValueError, match="format"):
        G.quantize_fp4(x, "fp5")
    with pytest.raises(TypeError):
        G.quantize_fp4(x.half())
    with pytest.raises(ValueError, match="dense rows"):
        G.quantize_fp4(torch.zeros((64, 64), device=DEV).t())
    lhs = G.quantize_fp4(x)
    rhs = G.quantize_fp4(torch.zeros((2, 16, 64), dtype=torch.bfloat16, device=DEV))
    gs = torch.tensor([2, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="mxfp4"):
        G.gmm_fp4(G.quantize_fp4(x, "mxfp4"), rhs, gs)
    with pytest.raises(ValueError, match="k="):
        G.gmm_fp4(G.quantize_fp4(x[:, :32]), rhs, gs)
    with pytest.raises(ValueError, match="row_scale"):
        G.gmm_fp4(lhs._replace(row_scale=None), rhs, gs)
    with pytest.raises(ValueError, match="block_scale"):
        G.gmm_fp4(lhs._replace(block_scale=lhs.block_scale[:, :2].contiguous()), rhs, gs)
    with pytest.raises(TypeError, match="group_sizes"):
        G.gmm_fp4(lhs, rhs, gs.long())
    with pytest.raises(G.GmmError, match="group_offset"):
        G.gmm_fp4(lhs, rhs, gs, group_offset=1)
    with pytest.raises(G.GmmError, match="unsupported sizes"):
        G.gmm_fp4(lhs, G.quantize_fp4(torch.zeros((2, 12, 64), dtype=torch.bfloat16, device=DEV)), gs)
    with pytest.raises(G.GmmError, match="workspace"):
        G.gmm_fp4(lhs, rhs, gs, workspace=torch.zeros(128, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="out must be"):
        G.gmm_fp4(lhs, rhs, gs, out=torch.zeros((4, 8), device=DEV))
    with pytest.raises(ValueError, match="rhs_bias"):
        G.gmm_fp4(lhs, rhs, gs, rhs_bias=torch.zeros((2, 16), device=DEV))


@pytest.mark.parametrize("groups,first,count", [(1024, 0, 1024), (1000, 37, 500), (33, 1, 32), (5, 4, 1)])
def test_many_groups(groups, first, count):
    """As many groups as there can be, most of them of a few rows or none, and slices of them."""
    rng = np.random.default_rng(groups)
    sizes = rng.integers(0, 4, groups)
    sizes[rng.integers(0, groups, 3)] = 70
    k, n, m = 64, 32, int(sizes.sum())
    lhs, a = operand((m, k), "mxfp4", 14)
    rhs, w = operand((count, n, k), "mxfp4", 15)
    out = G.gmm_fp4(lhs, rhs, torch.tensor(sizes, dtype=torch.int32, device=DEV), group_offset=first,
                    out_dtype=torch.float32)
    assert G.read_device_errors() == 0
    check_product(out, a, w, sizes, first, None, k)
