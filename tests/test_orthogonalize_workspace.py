"""The workspace of sar_orthogonalize for matrices of up to 128 rows (or columns) and 4096 columns, whose iteration runs in
shared memory and needs none: its size does not grow with theirs."""
import pytest
import torch

from tests import block_ref as bref
from tests import operator_ref as ref

SHAPES = [(65535, 16, 16), (64, 16, 4096), (4096, 64, 64), (1, 128, 4096), (3, 4096, 128), (1, 1, 1)]


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_size_of_small_matrices(sar, batch, rows, cols):
    assert 0 < sar.sar_orthogonalize_workspace_bytes(batch, rows, cols) <= 256


def test_sizes_on_both_sides(sar):
    """From 129 rows or 4097 columns on two X, A and the polynomial lie there: twice four bytes an element at least."""
    size = sar.sar_orthogonalize_workspace_bytes
    for rows, cols in ((129, 129), (129, 4096), (128, 4097), (4097, 128)):
        assert size(1, rows, cols) >= 8 * rows * cols and size(2, rows, cols) >= 2 * 8 * rows * cols
    assert size(65536, 16, 16) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("batch,rows,cols", [(700, 16, 16), (64, 16, 4096), (3, 4096, 128), (9, 100, 700)])
def test_small_matrices_without_more(sar, batch, rows, cols):
    g = torch.randn(batch, rows, cols, generator=torch.Generator(device="cuda").manual_seed(rows), device="cuda")
    out, again = torch.empty_like(g), torch.empty_like(g)
    ws = torch.full((256 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sar.sar_orthogonalize(g, out, ws[:256])
    sar.sar_orthogonalize(g, again, torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, again) and bool((ws[256:] == 0xA5).all())
    want, bound = bref.newton_schulz_bound(g, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    off = (out.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert bool((off <= bound + ref.U).all())
