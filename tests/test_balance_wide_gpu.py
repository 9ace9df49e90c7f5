"""balance_loss() and its gradient with many experts and enough tokens for sums that several CTAs join: every number of
experts a lane holds, in one cluster and in many, against the 64-bit statement and its bounds."""

import pytest
import torch

from test_balance_gpu import check, make

pytestmark = pytest.mark.gpu

# tokens, experts, topk, sequences: from 33 to 1024 experts, in one cluster of 16 CTAs (up to 2048 tokens), several, and
# clusters of each sequence
SHAPES = [(600, 1024, 8, 1), (2048, 1000, 4, 1), (5000, 513, 8, 1), (2048, 1024, 1, 1), (4099, 1024, 2, 1), (1023, 300, 3, 1),
          (6000, 520, 4, 3), (1200, 999, 6, 12), (2048, 40, 4, 1), (3000, 100, 4, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_losses_loads_and_gradient(shape, dtype, score):
    tokens, experts, topk, sequences = shape
    logits, chosen = make(tokens, experts, topk, dtype, tokens + experts)
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(5)) > 0.2
    check(logits, chosen, score, None, sequences)
    check(logits, chosen, score, mask, sequences, pitch=5)
