"""sar_expert_layer without hidden values: zeros, whatever the weights."""
import math

import pytest
import torch

from tests.test_gpu_expert_layer import case, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("tokens,topk,experts,cols", [(3, 2, 4, 16), (70, 3, 2, 33)])
def test_zeros_whatever_the_weights(sar, tokens, topk, experts, cols, dtype):
    x, _, w_in, w_out, weights = case(tokens, topk, experts, cols, 0, dtype, seed=2)
    ids = torch.zeros(tokens, topk, dtype=torch.int32, device="cuda")
    weights[0, 0], weights[1, 1], weights[2, 0] = math.inf, math.nan, -math.inf
    assert not layer(sar, x, ids, w_in, w_out, weights).any()
