"""dequantize_fp4() with row scales of any value: each value of the 64-bit product rounded once to the output's
type, bit for bit."""

import numpy as np
import pytest
import torch

import moe_grouped_matrix_gb300 as G
import moe_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rounded(v, dtype):
    """v in 64 bits rounded once to the type's values, ties to even (R._to_bits's spacing for magnitudes)."""
    bits, top = (7, 2.0 ** 128 * (1 - 2.0 ** -9)) if dtype == torch.bfloat16 else (23, 2.0 ** 128 * (1 - 2.0 ** -25))
    m = R._to_bits(np.abs(v), bits, -126)
    return np.copysign(np.where(np.abs(v) >= top, np.inf, m), v)


def check(codes, byte, row, dtype):
    q = G.Fp4Tensor(torch.from_numpy(R.pack(codes)).to(DEV), torch.from_numpy(R.to_windows(byte)).to(DEV),
                    torch.from_numpy(row).to(DEV), "nvfp4")
    got = G.dequantize_fp4(q, dtype).double().cpu().numpy()
    v = R.values(codes, byte, None, "nvfp4") * row.astype(np.float64)[:, None]
    np.testing.assert_array_equal(got, rounded(v, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_that_fp32_rounds_onto_a_half_way_point(dtype):
    """Row scales a third of a point half way between two bf16 values, rounded to fp32: three times them is
    off the point, in fp32 it is the point itself."""
    half = (256 + np.arange(128) * 2 + 1) * 2.0 ** -9  # odd multiples of half the spacing in [0.5, 1)
    row = np.concatenate([(h / 3).astype(np.float32) * s for h in (half, half * 2.0 ** -60, half * 2.0 ** 90)
                          for s in (np.float32(1), np.float32(-1))])
    off = 3.0 * row.astype(np.float64)
    assert (off.astype(np.float32).astype(np.float64) != off).mean() > 0.5
    codes = np.tile(np.array([5, 13, 2, 10, 4, 7, 1, 3], np.uint8), (len(row), 4))  # 3, -3, 1, -1, 2, 6, 0.5, 1.5
    check(codes, np.full((len(row), 2), 0x38, np.uint8), row, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_scales_of_any_value(dtype):
    rng = np.random.default_rng(0)
    rows, k = 300, 4096
    row = (rng.standard_normal(rows) * np.exp2(rng.integers(-120, 100, rows))).astype(np.float32)
    row[:8] = [0.0, 1.0, -2.0, 2.0 ** -126, 2.0 ** -140, 3e38, 1e-45, 1.1754942e-38]
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    byte = rng.integers(0, 127, (rows, k // 16)).astype(np.uint8)
    check(codes, byte, row, dtype)
