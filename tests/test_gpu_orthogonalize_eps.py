"""eps of sar_orthogonalize that is far above the gradient's norm."""
import pytest
import torch

from tests.test_gpu_orthogonalize import check, gradients

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("rows,cols", [(40, 64), (140, 150)])
@pytest.mark.parametrize("size,eps,steps", [(1e-15, 1e14, 20), (1e-15, 1e15, 30), (1e-14, 1e15, 50), (1e-20, 1e16, 40), (1e-13, 1e24, 60), (1e-3, 1e30, 40), (1e-3, 1e34, 45), (1e-4, 1e36, 50), (1e-2, 1e38, 63), (1e15, 1e38, 30)])
def test_eps_beside_any_gradient(sar, rows, cols, size, eps, steps):
    """X begins 1e-23 to 1e-40 in size and grows by 3.4445 a step."""
    check(sar, gradients(2, rows, cols, torch.float32, seed=5, scale=size), steps=steps, eps=eps)
