"""Clusters of blocks that each take a SM's tensor memory (sar_orthogonalize of up to 128 rows), many of them at once on
streams of their own, beside single blocks and the general form."""
import pytest
import torch

from tests.test_gpu_orthogonalize import check, gradients, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,rows,cols", [(100, 20, 257), (70, 128, 300), (60, 700, 33), (40, 64, 1030), (30, 8, 2100), (25, 128, 4096)])
def test_more_clusters_than_fit(sar, batch, rows, cols, dtype):
    check(sar, gradients(batch, rows, cols, dtype, seed=rows + cols))


def test_clusters_of_many_calls(sar):
    gs = [gradients(*shape, dtype, i) for i, (shape, dtype) in enumerate([
        ((80, 128, 300), torch.float32), ((60, 64, 1000), torch.bfloat16), ((30, 4096, 128), torch.float32), ((300, 64, 64), torch.float16),
        ((50, 60, 128), torch.float32), ((20, 128, 2000), torch.float16), ((2, 300, 500), torch.float32)])]
    want = [run(sar, g) for g in gs]
    outs = [torch.empty_like(g) for g in gs]
    spaces = [torch.empty(sar.sar_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device="cuda") for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, out, ws, s in zip(gs, outs, spaces, streams):
            sar.sar_orthogonalize(g, out, ws, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)
