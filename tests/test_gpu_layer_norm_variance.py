"""Layer norm of nearly constant rows far from zero: the sum of squares around
the mean is joined from the warps' parts, whose sums are rounded, and must not
come out below zero."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_layer_norm import forward

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


# Rows of one warp, of several, with two and with four vectors a thread in the kernel for many rows; then few rows, over
# each number of warps.
SHAPES = [(38912, 80), (39001, 127), (12160, 376), (5000, 1000), (330, 3000), (310, 5001), (320, 8000),
          (900, 130), (1100, 376), (300, 1000), (150, 2500), (140, 4092), (700, 1000), (250, 4000), (60, 7000), (20, 30000)]


@pytest.mark.parametrize("spread", ["constant", "one ulp"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_nearly_constant_rows(sar, shape, spread):
    """With e the bound of the mean: each warp's mean and the joined one are off by e at most, so that its squares around
    its own mean are over by e^2, and moving them costs up to (2 e)^2 and twice 2 e times e: 9 e^2 in all.  Below, there
    is no variance less than zero."""
    rows, cols = shape
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (10 ** (4 + 3 * torch.rand(rows, 1, generator=g, device="cuda", dtype=torch.float64))).float().repeat(1, cols)
    if spread == "one ulp":
        up = torch.nextafter(x, torch.full_like(x, float("inf")))
        x = torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.5, up, x)
    y, mean, rstd = forward(sar, x, None, None, EPS)
    (_, wm, _), (_, bm, _) = ref.layer_norm(x, None, None, EPS)
    ref.check(mean, wm, bm, "mean")
    d = x.double() - wm[:, None]
    var = (d * d).mean(1)
    assert bool(torch.isfinite(rstd).all()) and bool(torch.isfinite(y).all())
    low = 1 / torch.sqrt((1 + (ref.row_depth(cols) + 8) * ref.U) * var + 9 * bm ** 2 + EPS)
    assert bool((rstd.double() >= low * (1 - 4 * ref.U)).all())
    assert bool((rstd.double() <= EPS ** -0.5 * (1 + 4 * ref.U)).all())
    assert bool((y.double().abs() <= (d.abs() + bm[:, None]) * rstd.double()[:, None] * (1 + 4 * ref.U)).all())
