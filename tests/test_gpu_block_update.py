"""Steps of the block with experts over simulated ranks, each followed by the update of the parameters from the summed
gradients (allreduce_reduction_rank_gb300.block_step): router, sort, dispatch, combine, their gradients, the allreduce and
the orthogonalisation together."""
import pytest
import torch

from tests import block_ref as bref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,tokens,cols,experts,topk", [(2, 60, 64, 4, 2), (3, 150, 160, 6, 3)])
def test_steps_and_updates(ranks, tokens, cols, experts, topk):
    from allreduce_reduction_rank_gb300 import block_step as B
    params = B.Parameters.random(cols, experts, torch.float32, seed=5)
    steps, update = [B.RankStep(tokens, params, topk) for _ in range(ranks)], B.Update(params, rate=0.1)
    g = torch.Generator(device="cuda").manual_seed(6)
    for _ in range(3):                                  # parameters move, buffers are used again
        xs, dys = ([torch.randn(tokens, cols, generator=g, device="cuda") for _ in steps] for _ in range(2))
        ys, dxs, sums = B.step(steps, xs, dys)
        want = [B.reference(params, x, dy, s.ids) for x, dy, s in zip(xs, dys, steps)]
        # as test_gpu_block_step: 20 units of a chain of roundings, 16 for sums that cancel
        assert all(B.deviation(y, w[0]) < 20 * 16 * 2.0 ** -24 for y, w in zip(ys, want))
        assert B.deviation(sums[0], sum(w[2] for w in want)) < 20 * 16 * 2.0 ** -24
        for s in steps:                                 # what the router chose: the best scores, in order
            best = torch.topk(s.scores, topk, dim=1)
            assert torch.equal(best.values, s.scores.gather(1, s.ids))
            assert ((s.weights - torch.softmax(best.values, 1)).abs().max()) < 1e-6
        before = [p.clone() for p in (params.norm_weight, params.norm_bias, params.router, params.experts)]
        update.apply(params, sums[0])
        parts = torch.split(sums[0], [b.numel() for b in before])
        for b, p, d in zip(before, (params.norm_weight, params.norm_bias, params.router, params.experts), parts):
            if b.dim() == 1:
                assert torch.equal(p, b - 0.1 * d)
                continue
            scale = max(1.0, cols / experts) ** 0.5 if b.dim() == 2 else 1.0
            moved, bound = bref.newton_schulz_bound(d.view(b.shape) if b.dim() == 3 else d.view(1, *b.shape), 5,
                                                    (3.4445, -4.7750, 2.0315), 1e-7, scale)
            off = ((b - p).double() - 0.1 * moved.view(b.shape)).flatten().norm() / (0.1 * moved).flatten().norm()
            # the parameters' own rounding: half a unit of |p| beside a step of 0.1
            assert off <= bound.max() + 2.0 ** -23 * p.double().norm() / (0.1 * moved).flatten().norm()


def test_the_command_runs(capsys, monkeypatch):
    from allreduce_reduction_rank_gb300 import block_step as B
    monkeypatch.setattr("sys.argv", ["block_step", "--ranks", "2", "--tokens", "40", "--cols", "64", "--experts", "4"])
    B.main()
    assert "update: router" in capsys.readouterr().out
