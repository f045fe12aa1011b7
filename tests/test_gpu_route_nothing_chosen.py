"""The router's gradient where a token has chosen no expert, or has nothing to choose from: zeros, whatever its logits."""
import math

import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_route import MODES, backward, check_backward, scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@MODES
@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("experts", [5, 64, 300, 1024])
def test_no_chosen_expert_gives_zeros(sar, experts, dtype, every):
    inf, nan, d = math.inf, math.nan, ref.DTYPES[dtype]
    x = scores(8, experts, torch.float32, experts)
    x[0, 1] = nan
    x[1, 2], x[2, 0] = inf, -inf
    x[3] = -inf
    x[4, 3], x[4, 4] = inf, nan
    x[5] = nan
    x = x.to(d)
    dw = torch.randn(8, 4, generator=torch.Generator().manual_seed(experts)).cuda()
    ids = torch.tensor([[-1] * 4, [experts] * 4, [-1, experts, -2, 2 ** 31 - 1], [-1] * 4, [-1] * 4, [-5] * 4, [-1] * 4,
                        [1, -1, 4, 1]], device="cuda")
    for given in (ids, ids.int()):
        for dweights in (dw, torch.where((ids >= 0) & (ids < experts), dw, nan)):        # dropped ones are never read
            got = backward(sar, dweights, x, given, every)
            assert not got[:7].any() and not torch.isnan(got).any()
            assert got[7].any()
    check_backward(sar, dw[6:], x[6:], ids[6:], every)


@MODES
def test_masked_choices_beside_none(sar, every):
    """Minus infinity for all of a token's logits, or (softmax over the chosen) for all that it chose."""
    x = torch.full((3, 40), -math.inf, device="cuda")
    x[2, 7] = 1.0
    ids = torch.tensor([[3, 4], [-1, 39], [5, 6]], device="cuda")
    got = backward(sar, torch.ones(3, 2, device="cuda"), x, ids, every)
    assert not got.any()
