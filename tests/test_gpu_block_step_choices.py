"""A rank's step of the block with experts (allreduce_reduction_rank_gb300.block_step): more choices a token than
sar_expert_route makes, and choices kept over the next step."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("topk", [32, 33, 48])
def test_many_choices(topk):
    """Bounds as in test_gpu_block_step: 20 units of a chain of roundings, 16 for sums that cancel."""
    from allreduce_reduction_rank_gb300 import block_step as B
    params = B.Parameters.random(64, 48, torch.float32, seed=7)
    steps = [B.RankStep(50, params, topk) for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(8)
    for _ in range(2):
        xs, dys = ([torch.randn(50, 64, generator=g, device="cuda") for _ in steps] for _ in range(2))
        ys, dxs, sums = B.step(steps, xs, dys)
        want = [B.reference(params, x, dy, s.ids) for x, dy, s in zip(xs, dys, steps)]
        unit = 2.0 ** -24 * 16
        assert all(B.deviation(y, w[0]) < 20 * unit and B.deviation(dx, w[1]) < 20 * unit for y, dx, w in zip(ys, dxs, want))
        assert B.deviation(sums[0], sum(w[2] for w in want)) < 20 * unit
        for s in steps:
            best = torch.topk(s.scores, topk, dim=1)
            assert s.ids.shape == (50, topk) and torch.equal(best.values, s.scores.gather(1, s.ids))


def test_the_command_takes_many_choices(capsys, monkeypatch):
    from allreduce_reduction_rank_gb300 import block_step as B
    monkeypatch.setattr("sys.argv", ["block_step", "--ranks", "2", "--tokens", "40", "--cols", "64", "--experts", "40", "--topk", "36"])
    B.main()
    assert "36 of 40 experts" in capsys.readouterr().out


@pytest.mark.parametrize("topk", [3, 40])
def test_choices_of_a_step_stay(topk):
    from allreduce_reduction_rank_gb300 import block_step as B
    step = B.RankStep(30, B.Parameters.random(64, 48, torch.float32, seed=9), topk)
    g = torch.Generator(device="cuda").manual_seed(10)
    step.forward(torch.randn(30, 64, generator=g, device="cuda"))
    ids, weights = step.ids, step.weights
    was = ids.clone(), weights.clone()
    step.forward(torch.randn(30, 64, generator=g, device="cuda"))
    assert torch.equal(ids, was[0]) and torch.equal(weights, was[1])
    assert not torch.equal(step.ids, ids) and not torch.equal(step.weights, weights)
