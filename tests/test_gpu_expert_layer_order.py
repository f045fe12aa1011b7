"""sar_expert_layer's second kernel reads the ids before it waits for the first: calls that follow one another over the same
buffers, without anything between them, see their own ids."""
import pytest
import torch

from tests.test_gpu_expert_layer import case, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", [(1, 4, 16, 256, 96), (12, 3, 8, 128, 64), (40, 2, 8, 136, 72)])
@pytest.mark.parametrize("graph", [False, True], ids=["stream", "graph"])
def test_router_and_layer_in_turn(sar, tokens, topk, experts, cols, hidden, graph):
    count = 60
    x, _, w_in, w_out, _ = case(tokens, topk, experts, cols, hidden, "bf16", seed=cols)
    logits = torch.randn(count, tokens, experts, generator=torch.Generator().manual_seed(tokens)).cuda()
    ids, weights = torch.empty(tokens, topk, dtype=torch.int32, device="cuda"), torch.empty(tokens, topk, device="cuda")
    ws = torch.empty(sar.sar_expert_layer_workspace_bytes(tokens, topk, experts, cols, hidden), dtype=torch.uint8, device="cuda")
    outs = torch.empty(count, tokens, cols, dtype=x.dtype, device="cuda")

    def run():
        for i in range(count):
            sar.sar_expert_route(logits[i], ids, weights)
            sar.sar_expert_layer(x, ids, w_in, w_out, outs[i], weights, workspace=ws)
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        for _ in range(3):
            g.replay()
    else:
        run()
    torch.cuda.synchronize()
    for i in range(count):
        mine = torch.empty_like(ids), torch.empty_like(weights)
        sar.sar_expert_route(logits[i], *mine)
        torch.cuda.synchronize()
        assert torch.equal(outs[i], layer(sar, x, mine[0], w_in, w_out, mine[1])), i
