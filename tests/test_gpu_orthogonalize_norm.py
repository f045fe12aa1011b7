"""The norm of sar_orthogonalize over matrices of values of one magnitude, the squares' hardest sum: additions of one term
again and again err to one side."""
import pytest
import torch

from tests import operator_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("value", [1.4707840, 0.6864250])
@pytest.mark.parametrize("rows,cols,gap", [(4096, 65536, 0), (4096, 65535, 1), (65536, 2048, 0), (300, 65521, 0), (128, 4096, 0),
                                           (2049, 100, 3)])
def test_norm_of_equal_magnitudes(sar, rows, cols, gap, value):
    """With the polynomial s the result is g / |g|, every element rows cols ^ -1/2 in magnitude.  The sum of squares: up to
    64 additions of a few terms, joined with a compensated sum, 16 more in a block and 16 for the blocks' sums, U each;
    half of that for its root, and 8 U for the root, the reciprocal and the products."""
    g = torch.empty(rows, cols + gap, device="cuda")[:, :cols]
    signs = torch.rand(rows, cols, generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda") < 0.5
    g.copy_(torch.where(signs, value, -value))
    out = torch.empty_like(g)
    ws = torch.empty(sar.sar_orthogonalize_workspace_bytes(1, rows, cols), dtype=torch.uint8, device="cuda")
    sar.sar_orthogonalize(g, out, ws, steps=1, coefficients=(1.0, 0.0, 0.0), eps=0.0)
    assert torch.equal(out > 0, signs)
    size = out.abs_()
    want, low, high = (rows * cols) ** -0.5, size.min().item(), size.max().item()
    assert max(abs(low / want - 1), abs(high / want - 1)) <= ref.SLACK * ((64 + 32) / 2 + 8) * ref.U
