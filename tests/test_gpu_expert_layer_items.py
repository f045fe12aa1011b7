"""The expert layer (sar_expert_layer) on both sides of each switch of an item's slots: by the slots that an expert has on
average, 4, 6, 10 and 20 and one more."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_expert_layer import case, check_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("cols,hidden", [(64, 48), (72, 37), (67, 64), (45, 83)])
@pytest.mark.parametrize("mean", [4, 5, 6, 7, 10, 11, 20, 21, 40])
def test_slots_of_an_expert(sar, mean, cols, hidden, dtype):
    x, ids, w_in, w_out, weights = case(mean * 3, 2, 6, cols, hidden, dtype, seed=mean + cols)
    check_layer(sar, x, ids, w_in, w_out, weights)
    uneven = torch.where(ids > 3, 0, ids)                     # one expert has three times the others' and a token has it twice
    check_layer(sar, x, uneven, w_in, w_out, weights, gap=1)
