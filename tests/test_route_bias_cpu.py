"""gmm_route()'s score argument with and without GMM_SCORE_BIASED (no GPU needed; no pointer is followed)."""

import ctypes

import pytest

import moe_grouped_matrix_gb300 as G
from moe_grouped_matrix_gb300 import build as B

P, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)
SHAPE, ALIGN = 3, 4


@pytest.fixture(scope="module")
def lib():
    B.build()
    return G.load_library()


def test_the_scores_that_are_taken(lib):
    for score in (-1, 0, 1, 2, 15, 16, 17, 18, 32, 33):
        status = lib.gmm_route(P, 1, 4, 8, 8, 2, score, 1, 1.0, P, None, P, ODD, None)
        assert status == (ALIGN if score in (0, 1, 16, 17) else SHAPE), score
        status = lib.gmm_route_backward(P, P, P, 1, 4, 8, 8, 2, score, 1, 1.0, ODD, None)
        assert status == (ALIGN if score in (0, 1) else SHAPE), score
