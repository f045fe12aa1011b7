"""The gradient of layer norm at the ends of binary32's range: what the formula
keeps finite, or keeps at all, the kernels do too."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_layer_norm import backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def check(sar, dy, x, w, mean, rstd, gap=0, offset=0):
    dx, dw, db = backward(sar, dy, x, w, mean, rstd, torch.float32, gap, offset)
    (wx, ww, wb), (bx, bw, bb) = ref.layer_norm_backward(dy, x, w, mean, rstd)
    ref.check(dx, wx, ref.rounded(bx, wx, x.dtype), "dx")
    ref.check(dw, ww, ref.rounded(bw, ww, torch.float32), "dweight")
    ref.check(db, wb, ref.rounded(bb, wb, torch.float32), "dbias")


# Few rows and many, of one, two and four vectors a thread, whole and off 16-byte boundaries.
SHAPES = [(40, 1024), (9, 1021), (24400, 128), (3100, 1024), (3100, 1021), (330, 4096), (330, 5003), (330, 8192)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_of_tiny_spread(sar, shape, dtype):
    """Rows of spread 1e-20 and eps = 0: rstd is 1e20, whose square is no binary32 value."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64) * 1e-20).to(ref.DTYPES[dtype])
    dy = torch.randn(*shape, generator=g, device="cuda").to(x.dtype)
    w = 1 + 0.2 * torch.randn(shape[1], generator=g, device="cuda")
    d = x.double() - x.double().mean(1, keepdim=True)
    check(sar, dy, x, w, x.double().mean(1).float(), (d * d).mean(1).rsqrt().float())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows_of_huge_spread(sar, shape, dtype):
    """Rows of spread 1e18 whose gradient lies along them and is small: rstd^2 mean(g h) is 1e-46, less than any binary32
    value, but the term that it belongs to is the largest of dx."""
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float64)
    x = (h * 1e18).to(ref.DTYPES[dtype])
    dy = (1e-10 * (h + 0.3 * torch.randn(*shape, generator=g, device="cuda"))).to(x.dtype)
    w = 1 + 0.2 * torch.randn(shape[1], generator=g, device="cuda")
    d = x.double() - x.double().mean(1, keepdim=True)
    check(sar, dy, x, w, x.double().mean(1).float(), (d * d).mean(1).rsqrt().float())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gap,offset", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("shape", [(5, 37), (7, 100), (9, 136), (40, 250), (3, 1021), (3, 1500), (24400, 100), (24400, 136),
                                   (39000, 250), (3100, 1020), (7300, 1021), (330, 5000), (330, 5003)], ids=str)
def test_constant_rows_of_a_great_value(sar, shape, gap, offset, dtype):
    """Rows of 2^110 throughout with eps = 1e-12: h is 0 and dx = rstd (g - mean(g)) with rstd = 1e6.  A place past the
    row's end, which holds 0, would have (0 - mean) rstd = -infinity."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.full(shape, 2.0 ** 110, device="cuda", dtype=ref.DTYPES[dtype])
    dy = torch.randn(*shape, generator=g, device="cuda").to(x.dtype)
    mean = torch.full(shape[:1], 2.0 ** 110, device="cuda")
    check(sar, dy, x, None, mean, torch.full_like(mean, 1e6), gap, offset)
