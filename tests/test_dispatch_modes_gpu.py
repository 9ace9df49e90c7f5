"""PyTorch's dispatch modes see the results that the MoE operators allocate, and tensors of a subclass go
the way on which each of their operations is asked for."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from test_moe_streams_gpu import CALLS, data, same  # noqa: F401

pytestmark = pytest.mark.gpu
RESULTS = {"route": 2, "route_sigmoid": 2, "route_backward": 1, "sort_by_expert": 3, "dispatch": 1,
           "dispatch_backward": 1, "combine": 1, "combine_backward": 2, "quantize": 3, "quantize_order": 2,
           "dequantize": 1, "gmm_fp4": 1, "gmm_fp4_mx": 1}


class Allocations(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.count = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.count += func in (torch.ops.aten.empty.memory_format, torch.ops.aten.empty_like.default)
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_mode_sees_the_results(data, name):  # noqa: F811
    want = CALLS[name](data)
    with Allocations() as seen:
        got = CALLS[name](data)
    assert seen.count == RESULTS[name]
    assert same(got, want)
