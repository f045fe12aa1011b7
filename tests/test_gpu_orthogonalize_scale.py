"""The largest and smallest scales of sar_orthogonalize: the result leaves binary32's range only where the formula does."""
import pytest
import torch

from tests.test_gpu_orthogonalize import check, gradients, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("rows,cols", [(40, 64), (140, 150), (260, 900)])
@pytest.mark.parametrize("scale", [3e38, -1e36, 1e34, 2.0 ** 120, 1e-30, 2.0 ** -120, 0.0])
def test_scales(sar, rows, cols, scale):
    g = gradients(2, rows, cols, torch.float32, seed=3)
    plain = run(sar, g)
    got = run(sar, g, scale=scale)
    # one product, rounded once, of plain's elements: what is below a power of two is lost where it is subnormal
    assert torch.equal(got.double(), (plain.double() * torch.tensor(scale).double()).float().double()) if scale not in (1e-30, 2.0 ** -120) \
        else bool(((got.double() - plain.double() * torch.tensor(scale).double()).abs() <= 2.0 ** -24 * got.abs().double() + 2.0 ** -149).all())


@pytest.mark.parametrize("rows,cols", [(40, 64), (140, 150)])
def test_a_large_scale_of_what_is_small(sar, rows, cols):
    """eps beside which the gradient vanishes: X of 1e-30, scaled by 1e36."""
    check(sar, gradients(2, rows, cols, torch.float32, seed=4, scale=1e-6), steps=3, eps=1e24, scale=1e36)
