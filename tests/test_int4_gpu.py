"""Weights in 4-bit integers, and their products with few tokens, against the 64-bit statement.

Codes, scales and zero points are decided by exact quotients and have to be equal.  A product is the sum
of scale code x and -scale zero x, codes counted from 0; it is off by at most experts_reference.matvec_adds() units of
2^-23 of the sum of these terms' sizes, its output by half a step."""

import numpy as np
import pytest
import torch

import experts_reference as R
import moe_grouped_matrix_gb300 as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BOTH = [False, True]


def normal(shape, seed, std=1.0, dtype=torch.float32):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (std * torch.randn(shape, generator=gen, device=DEV)).to(dtype)


# ---------------------------------------------------------------- quantisation
def check_quantize(x, group, zero_points):
    q = G.quantize_int4(x, group, zero_points)
    torch.cuda.synchronize()
    k = x.shape[-1]
    assert q.codes.shape == x.shape[:-1] + (k // 2,) and q.group == group and (q.zero is None) == (not zero_points)
    codes, scale, zero = R.quantize_int4(R.as64(x), group, zero_points)
    got_codes, got_scale, got_zero = R.unpack(q)
    np.testing.assert_array_equal(got_scale, scale)
    if zero_points:
        np.testing.assert_array_equal(got_zero, zero)
    np.testing.assert_array_equal(got_codes, codes)
    last = k % 256
    if last:  # entries past the last group
        assert not q.scale[..., -1, :, last // group:].any()
        assert zero is None or not q.zero[..., -1, :, last // group:].any()
    for dtype in (torch.float32, torch.bfloat16):
        v = G.dequantize_int4(q, dtype)
        assert v.shape == x.shape and v.dtype == dtype
        want = torch.from_numpy(R.values(q)).to(dtype)  # exact in 64 bits: rounded once
        assert torch.equal(torch.nan_to_num(v.cpu().float(), 7e7), torch.nan_to_num(want.float(), 7e7))
    return q


SHAPES = [(1, 128), (3, 256), (8, 384), (17, 1280), (5, 4096), (301, 640), (1, 16384), (5000, 256)]


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize(shape, dtype, group, zero_points):
    check_quantize(normal(shape, shape[1] + group, 0.02, dtype), group, zero_points)


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group,k", [(32, 32), (32, 96), (32, 288), (64, 64), (64, 448)])
def test_quantize_short_rows_batches_and_pitches(group, k, zero_points):
    check_quantize(normal((3, 9, k), k), group, zero_points)
    for offset, pitch in ((0, k + 8), (1, k + 1), (2, k + 4)):
        check_quantize(normal((9 * pitch + 8,), k)[offset:].as_strided((9, k), (pitch, 1)), group, zero_points)


@pytest.mark.parametrize("zero_points", BOTH)
def test_quantize_half_way_points(zero_points):
    """Every multiple of half a step and its neighbours in fp32, for scales of all 8-bit significands."""
    s = (torch.arange(128, 256, dtype=torch.float32, device=DEV) / 128)[:, None]
    h = torch.arange(-15, 16, dtype=torch.float32, device=DEV)[None] / 2 if not zero_points else \
        torch.arange(0, 31, dtype=torch.float32, device=DEV)[None] / 2 - 4
    x = torch.zeros((128, 128), device=DEV)
    for j, to in enumerate((-float("inf"), None, float("inf"))):
        v = s * h
        x[:, 31 * j:31 * (j + 1)] = v if to is None else torch.nextafter(v, torch.full_like(v, to))
    # the largest magnitude (spread) makes the scale s again: 7 s (15 s)
    if zero_points:
        x[:, 126:], x[:, 125:126] = -4 * s, 11 * s
        x.clamp_(min=-4 * s, max=11 * s)
    else:
        x[:, 127:] = 7 * s
        x.clamp_(min=-7 * s, max=7 * s)
    q = check_quantize(x, 128, zero_points)
    assert torch.equal(q.scale.float().reshape(-1, 2)[:, :1], s)


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", [32, 128])
def test_quantize_odd_values(group, zero_points):
    x = normal((16, 512), 3)
    x[0] = 0
    x[1, 5], x[2, 200], x[3, 100] = float("nan"), float("inf"), -float("inf")
    x[4] *= 1e-38
    x[5] *= 1e-42
    x[6] = x[6].abs()
    x[7] = -x[7].abs()
    x[8] = 1e-45
    x[9, 0], x[9, 1] = 3e38, -3e38
    x[10] *= 1e37
    x[11] = 5.0
    x[12] = torch.finfo(torch.float32).max
    x[13] *= 2.0 ** -101
    q = check_quantize(x, group, zero_points)
    w = G.dequantize_int4(q, torch.float32)
    assert w[1, :group].isnan().all() and not w[1, 128:].isnan().any() and not w[0].any()


@pytest.mark.parametrize("zero_points", BOTH)
def test_quantize_nothing(zero_points):
    q = G.quantize_int4(torch.empty((0, 256), device=DEV), 64, zero_points)
    assert q.codes.shape == (0, 128) and G.dequantize_int4(q).shape == (0, 256)
    q = G.quantize_int4(torch.empty((0, 4, 256), device=DEV), 64, zero_points)
    assert G.dequantize_int4(q).shape == (0, 4, 256)


# ---------------------------------------------------------------- products
def check_matvec(x, w, experts=None, weights=None, act=None, out_dtype=torch.float32, **more):
    out = G.matvec_int4(x, w, experts, weights, act, out_dtype, **more)
    torch.cuda.synchronize()
    assert out.dtype == out_dtype
    w64, sizes = R.values(w), R.term_sizes(w)
    if experts is None:
        want, size = R.matvec(R.as64(x), w64[None], np.zeros((x.shape[0], 1), int), None, act, sizes[None])
        want, size = want[:, 0], size[:, 0]
    else:
        want, size = R.matvec(R.as64(x), w64, experts.cpu().numpy(), None if weights is None else R.as64(weights), act,
                              sizes)
    assert tuple(out.shape) == want.shape
    tol = (R.matvec_adds(x.shape[-1], w.group) + x.shape[-1] // 256) * 2.0 ** -23 * size
    tol = tol + R.half_step(out_dtype) * (np.abs(want) + tol) + 2.0 ** -126
    assert (np.abs(R.as64(out) - want) <= tol).all()
    return out


def make(experts, n, k, group, zero_points, seed=1):
    return G.quantize_int4(normal((experts, n, k), seed, 0.05), group, zero_points)


def choose(tokens, experts, topk, seed, dropped=0.1):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    score = torch.rand((tokens, experts), generator=gen, device=DEV)
    chosen = torch.sort(score, dim=1, stable=True)[1][:, :topk].to(torch.int32)
    chosen[torch.rand(chosen.shape, generator=gen, device=DEV) < dropped] = -1
    return chosen.contiguous()


# tokens, experts, topk, n, k
CASES = [(1, 8, 2, 256, 256), (1, 1, 1, 8, 128), (2, 3, 3, 24, 384), (9, 4, 2, 40, 640), (17, 2, 1, 72, 1024),
         (33, 5, 4, 136, 2048), (5, 64, 8, 48, 4224), (40, 7, 7, 16, 256), (3, 1024, 32, 8, 128), (1, 2, 2, 2072, 512)]


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", CASES)
def test_products_by_slot(case, group, zero_points, out_dtype):
    tokens, E, topk, n, k = case
    w = make(E, n, k, group, zero_points)
    experts = choose(tokens, E, topk, k)
    out = check_matvec(normal((tokens, k), 2, dtype=torch.bfloat16), w, experts, out_dtype=out_dtype)
    assert not out[experts < 0].any()
    check_matvec(normal((tokens, topk, k), 3, dtype=torch.bfloat16), w, experts, out_dtype=out_dtype)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", [c for c in CASES if c[3] % 16 == 0])
def test_products_with_the_activation(case, group, zero_points, act):
    tokens, E, topk, n, k = case
    w = make(E, n, k, group, zero_points)
    check_matvec(normal((tokens, k), 2, dtype=torch.bfloat16), w, choose(tokens, E, topk, k), act=act)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("case", CASES)
def test_sums_over_the_slots(case, group, zero_points, out_dtype):
    tokens, E, topk, n, k = case
    w = make(E, n, k, group, zero_points)
    weights = normal((tokens, topk), 5)
    for x in (normal((tokens, topk, k), 3, dtype=torch.bfloat16), normal((tokens, k), 3, dtype=torch.bfloat16)):
        check_matvec(x, w, choose(tokens, E, topk, n), weights, out_dtype=out_dtype)


@pytest.mark.parametrize("zero_points", BOTH)
@pytest.mark.parametrize("tokens,n,k", [(1, 4096, 1024), (1, 16, 16384), (8, 200, 768), (13, 64, 2304)])
def test_one_matrix(tokens, n, k, zero_points):
    w = make(1, n, k, 64, zero_points)
    w = G.Int4Tensor(w.codes[0], w.scale[0], None if w.zero is None else w.zero[0], 64)
    check_matvec(normal((tokens, k), 2, dtype=torch.bfloat16), w)
    check_matvec(normal((tokens, k), 2, dtype=torch.bfloat16), w, act="silu") if n % 16 == 0 else None


# tokens, experts, topk, n, k, group, zero points: much work for each CTA, where an item's x is copied at a time;
# the whole of 8 columns, and fewer than that, and ends of k and n within a tile
@pytest.mark.parametrize("case", [(40, 8, 2, 4096, 2176, 128, False), (40, 8, 2, 4104, 2048, 64, True),
                                  (24, 4, 2, 4096, 4096, 32, True), (48, 8, 2, 4112, 2080, 32, False),
                                  (17, 9, 1, 2064, 4096, 64, False)])
@pytest.mark.parametrize("act", [None, "silu"])
def test_products_of_many_tokens(case, act):
    tokens, E, topk, n, k, group, zero_points = case
    if act is not None and n % 16:
        n += 8
    w = make(E, n, k, group, zero_points)
    experts = choose(tokens, min(E, 9), topk, k)
    check_matvec(normal((tokens, k), 2, dtype=torch.bfloat16), w, experts, act=act)


@pytest.mark.parametrize("tokens,topk", [(256, 1), (257, 1), (128, 2), (8, 32), (9, 32)])
def test_the_most_slots_of_a_launch(tokens, topk):
    w = make(40, 48, 256, 64, False)
    x, experts = normal((tokens, 256), 2, dtype=torch.bfloat16), choose(tokens, 40, topk, 3)
    check_matvec(x, w, experts)
    check_matvec(x, w, experts, normal((tokens, topk), 5))


def test_long_rows_of_several_tokens():
    w = make(3, 64, 16384, 128, False)
    check_matvec(normal((9, 16384), 2, dtype=torch.bfloat16), w, choose(9, 3, 2, 1))
    check_matvec(normal((9, 2, 16384), 2, dtype=torch.bfloat16), w, choose(9, 3, 2, 1), normal((9, 2), 5))


def test_more_slots_than_a_launch_takes():
    w = make(6, 32, 256, 32, True)
    x = normal((1030, 256), 2, dtype=torch.bfloat16)
    for topk in (1, 3):
        experts = choose(1030, 6, topk, topk)
        check_matvec(x, w, experts)
        check_matvec(x, w, experts, normal((1030, topk), 5))
    check_matvec(normal((90, 32, 256), 2, dtype=torch.bfloat16), w, choose(90, 6, 6, 1).repeat(1, 6)[:, :32].contiguous(),
                 normal((90, 32), 5))


def test_an_expert_chosen_more_than_once():
    w = make(4, 48, 512, 64, False)
    experts = torch.tensor([[1, 1, 1], [2, 1, 2], [-1, 3, 3], [0, 4, 9], [-1, -5, 2 ** 31 - 1], [1, 1, 0]],
                           dtype=torch.int32, device=DEV)
    x = normal((6, 3, 512), 3, dtype=torch.bfloat16)
    check_matvec(x, w, experts)
    out = check_matvec(x, w, experts, normal((6, 3), 5))
    assert not out[4].any()


def test_weights_of_absent_slots_and_rows_of_absent_experts_are_not_read():
    w = make(4, 48, 512, 64, False)
    experts = choose(11, 4, 3, 1, dropped=0.0)
    experts[::2, 1] = -1
    experts[experts == 3] = -1  # nobody chooses expert 3
    w.codes[3], w.scale[3] = 0x77, float("nan")
    weights, x = normal((11, 3), 5), normal((11, 3, 512), 3, dtype=torch.bfloat16)
    weights[experts < 0], x[experts < 0] = float("nan"), float("nan")
    out = G.matvec_int4(x, w, experts, weights, out_dtype=torch.float32)
    rows = G.matvec_int4(x, w, experts, out_dtype=torch.float32)
    assert out.isfinite().all() and rows.isfinite().all() and not rows[experts < 0].any()
    weights[experts < 0], x[experts < 0] = 0, 0
    w.scale[3] = 0
    check_matvec(x, w, experts, weights)


def test_nan_and_infinity_reach_only_their_own_slots():
    w = make(2, 32, 512, 128, True)
    x = normal((9, 512), 3, dtype=torch.bfloat16)
    x[4, 77], x[5, 300] = float("nan"), float("inf")
    experts = torch.tensor([[0, 1]] * 9, dtype=torch.int32, device=DEV)
    out = G.matvec_int4(x, w, experts, out_dtype=torch.float32)
    assert out[4].isnan().all() and not out[5].isfinite().any()
    rest = [0, 1, 2, 3, 6, 7, 8]
    assert torch.equal(out[rest], G.matvec_int4(x[rest], w, experts[rest], out_dtype=torch.float32))


@pytest.mark.parametrize("power", [-120, -60, 60, 110])
def test_rows_of_x_of_any_size(power):
    """Rows next to others that are far larger or smaller, and values in a row that span bf16's range."""
    w = make(3, 48, 768, 64, True)
    x = normal((10, 768), 3, dtype=torch.bfloat16)
    x[2:5] *= 2.0 ** power
    x[5, ::2] *= 2.0 ** power
    x[6, 1:] = 0
    x[7] = 0
    x[8] = torch.tensor([1, 3 - 2 ** 15], dtype=torch.int16, device=DEV).view(torch.bfloat16).repeat(384)  # subnormal
    experts = choose(10, 3, 2, 1, 0.0)
    check_matvec(x, w, experts)
    check_matvec(x.repeat(7, 1), w, experts.repeat(7, 1))
    weights = normal((10, 2), 4)
    check_matvec(x, w, experts, weights)


def test_entries_past_the_last_group_are_not_read():
    w = make(2, 32, 288, 32, True)
    x, experts = normal((3, 288), 3, dtype=torch.bfloat16), choose(3, 2, 2, 1, 0.0)
    want = check_matvec(x, w, experts)
    w.scale[:, 1, :, 1:], w.zero[:, 1, :, 1:] = float("nan"), 255
    assert torch.equal(want, G.matvec_int4(x, w, experts, out_dtype=torch.float32))


@pytest.mark.parametrize("pitch", [520, 1024, 4096])
def test_rows_with_a_pitch(pitch):
    w = make(3, 64, 512, 64, False)
    x = normal((12, pitch), 3, dtype=torch.bfloat16)[:, :512]
    experts = choose(12, 3, 2, 1)
    assert torch.equal(check_matvec(x, w, experts), G.matvec_int4(x.contiguous(), w, experts, out_dtype=torch.float32))


def test_no_tokens():
    w = make(3, 64, 512, 64, False)
    x, experts = torch.empty((0, 512), dtype=torch.bfloat16, device=DEV), torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert G.matvec_int4(x, w, experts).shape == (0, 2, 64)
    assert G.matvec_int4(x, w, experts, torch.empty((0, 2), device=DEV)).shape == (0, 64)
    assert G.matvec_int4(x, w, experts, act="silu").shape == (0, 2, 32)


def test_the_same_bits_again():
    w = make(16, 512, 2048, 128, False)
    x, experts = normal((7, 2048), 3, dtype=torch.bfloat16), choose(7, 16, 4, 1)
    weights = torch.rand((7, 4), device=DEV)
    first, rows = G.matvec_int4(x, w, experts, weights), G.matvec_int4(x, w, experts)
    for _ in range(30):
        assert torch.equal(first, G.matvec_int4(x, w, experts, weights))
        assert torch.equal(rows, G.matvec_int4(x, w, experts))


@pytest.mark.parametrize("zero_points", BOTH)
def test_a_layers_decoding_step(zero_points):
    """route() -> both products of the experts, against the layer of the values its weights stand for: the
    activations between are rounded to bf16 in both, at points that may differ by a rounding (2^-8 of each)."""
    T, E, K, d, f = 6, 16, 3, 512, 256
    x, router = normal((T, d), 1, dtype=torch.bfloat16), normal((E, d), 2, 0.05, torch.bfloat16)
    weights, experts = G.route(x @ router.T, K)
    wi, wo = make(E, 2 * f, d, 128, zero_points, 3), make(E, d, f, 64, zero_points, 4)
    h = G.matvec_int4(x, wi, experts, act="silu")
    y = G.matvec_int4(h, wo, experts, weights, out_dtype=torch.float32)
    e64 = experts.cpu().numpy()
    h64, _ = R.matvec(R.as64(x), R.values(wi), e64, None, "silu")
    y64, size = R.matvec(R.to_bf16(h64), R.values(wo), e64, R.as64(weights))
    assert (np.abs(R.as64(y) - y64) <= 2.0 ** -8 * size).all()
