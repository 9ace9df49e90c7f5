"""The largest sizes of the products: the kernels index rows, columns and depth in 32 bits and step up to a
tile past the last, so sizes within a tile of 2^31 are refused before anything is launched (no GPU needed;
no pointer is followed)."""

import ctypes

import pytest

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B

P = ctypes.c_void_p(1 << 20)
SHAPE, WORKSPACE = 3, 6
LARGEST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load_library()


def gmm(lib, m=64, k=64, n=64, dtype=0):
    return lib.gmm(P, 0, m, k, P, dtype, 4, n, 1, P, 4, 0, None, 0, None, 0, P, 0, None, 0, None)


def gmm_into(lib, m=64, k=64, n=64):
    return lib.gmm_into(P, 0, m, k, P, 0, 4, n, 1, P, 4, 0, None, 0, None, 0, P, 0, None, 0, None)


def tgmm(lib, m=64, k=64, n=64):
    return lib.tgmm(P, 0, P, 0, m, k, n, P, 4, P, 1, None, 0, None)


def gmm_fp4(lib, m=64, k=64, n=64):
    return lib.gmm_fp4(P, P, P, m, k, P, P, P, 0, 4, n, P, 4, 0, None, 0, P, 0, None, 0, None)


@pytest.mark.parametrize("call", [gmm, gmm_into, tgmm, gmm_fp4])
@pytest.mark.parametrize("size", ["m", "k", "n"])
def test_sizes_within_a_tile_of_2_to_the_31(lib, call, size):
    assert call(lib, **{size: LARGEST}) == WORKSPACE  # taken: what is refused is the missing workspace
    for more in (1, 8, 32, 768, 991, 992, 1000, 1016, 1023):
        if size == "m" or more % 32 == 0:
            assert call(lib, **{size: LARGEST + more}) == SHAPE, more
