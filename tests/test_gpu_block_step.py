"""The block with experts over simulated ranks (allreduce_reduction_rank_gb300.block_step): layer norm, sort, dispatch,
combine, their gradients and the allreduce together against torch.autograd in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# Relative deviations (2-norm): a chain of about ten roundings to the rows' type (h, rows, the product, the combine, the
# sum; and back), each of half the type's unit roundoff on average, and as much again for the terms that cancel in the
# sums over experts and tokens: 20 units.  fp32 products run without tf32.
@pytest.mark.parametrize("dtype,unit", [("bf16", 2.0 ** -8), ("fp16", 2.0 ** -11), ("fp32", 2.0 ** -24 * 16)])
@pytest.mark.parametrize("ranks,tokens,cols,experts,topk", [(1, 33, 64, 4, 2), (3, 200, 136, 8, 3), (2, 700, 256, 16, 1)])
def test_step_matches_autograd(ranks, tokens, cols, experts, topk, dtype, unit):
    from allreduce_reduction_rank_gb300 import block_step as B
    params = B.Parameters.random(cols, experts, B.TYPES[dtype], seed=3)
    steps = [B.RankStep(tokens, params, topk) for _ in range(ranks)]
    g = torch.Generator(device="cuda").manual_seed(4)
    for _ in range(2):                                  # buffers are used again
        xs, dys = ([torch.randn(tokens, cols, generator=g, device="cuda").to(B.TYPES[dtype]) for _ in steps] for _ in range(2))
        ys, dxs, sums = B.step(steps, xs, dys)
        want = [B.reference(params, x, dy, s.ids) for x, dy, s in zip(xs, dys, steps)]
        for y, dx, w in zip(ys, dxs, want):
            assert B.deviation(y, w[0]) < 20 * unit and B.deviation(dx, w[1]) < 20 * unit
        total = sum(w[2] for w in want)
        for s in sums:
            assert B.deviation(s, total) < 20 * unit and torch.equal(s, sums[0])
