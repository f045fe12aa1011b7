"""The router (sar_expert_route) and its gradient against one-token-at-a-time
and 64-bit definitions (tests/block_ref.py)."""
import math

import pytest
import torch

from tests import block_ref as bref
from tests import operator_ref as ref
from tests.test_gpu_layer_norm import MARK, placed, untouched

pytestmark = pytest.mark.gpu
MODES = pytest.mark.parametrize("every", [False, True], ids=["chosen", "all"])


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def scores(tokens, experts, dtype, seed=0, mask=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 1.5 * torch.randn(tokens, experts, generator=g, device="cuda")
    if mask:
        x[torch.rand(tokens, experts, generator=g, device="cuda") < mask] = -math.inf
        x[torch.rand(tokens, generator=g, device="cuda") < 0.2] = -math.inf
    return x.to(dtype)


def route(sar, x, topk, every, id_type=torch.int32, wdtype=torch.float32, gap=0, offset=0):
    tokens = x.shape[0]
    xv, _ = placed(x, gap, offset)
    ids = torch.full((tokens * topk + 2,), -77, dtype=id_type, device="cuda")
    weights = torch.full((tokens * topk + 2,), MARK, dtype=wdtype, device="cuda")
    sar.sar_expert_route(xv, ids[1:-1].view(tokens, topk), weights[1:-1].view(tokens, topk),
                         softmax=sar.SAR_SOFTMAX_ALL if every else sar.SAR_SOFTMAX_CHOSEN)
    torch.cuda.synchronize()
    assert int(ids[0]) == -77 and int(ids[-1]) == -77 and weights[0] == MARK and weights[-1] == MARK
    return ids[1:-1].view(tokens, topk), weights[1:-1].view(tokens, topk)


def check_route(sar, x, topk, every, **kw):
    ids, weights = route(sar, x, topk, every, **kw)
    want = bref.route(x, topk, every)
    assert ids.tolist() == want[0]
    ref.check(weights.cpu(), want[1], ref.rounded(want[2], torch.nan_to_num(want[1]), weights.dtype), "weights")


@MODES
@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("tokens,experts,topk,mask", [
    (1, 1, 1, 0.0), (1, 2, 2, 0.0), (3, 7, 3, 0.4), (9, 32, 8, 0.0), (8, 33, 1, 0.0), (32, 128, 8, 0.0), (17, 60, 6, 0.2),
    (100, 64, 32, 0.1), (13, 65, 16, 0.9), (50, 256, 8, 0.0), (7, 257, 12, 0.0), (33, 512, 8, 0.5), (5, 1000, 31, 0.0),
    (9, 1024, 32, 0.0), (1000, 16, 2, 0.0)])
def test_route(sar, tokens, experts, topk, mask, dtype, every):
    x = scores(tokens, experts, ref.DTYPES[dtype], tokens + experts, mask)
    check_route(sar, x, topk, every, gap=tokens % 3, offset=tokens % 2)
    check_route(sar, x, topk, every, id_type=torch.int64, wdtype=x.dtype)


@MODES
def test_equal_logits_take_the_lower_id(sar, every):
    x = torch.tensor([[0.0, -0.0, 0.0, -0.0], [1.0, 2.0, 2.0, 1.0], [5.0, 5.0, 5.0, 5.0], [-0.0, 0.0, -1.0, 1.0]], device="cuda")
    ids, _ = route(sar, x, 3, every)
    assert ids.tolist() == [[0, 1, 2], [1, 2, 0], [0, 1, 2], [3, 0, 1]]
    for experts in (40, 300, 1024):                       # coarse values: many ties
        check_route(sar, (scores(64, experts, torch.float32, experts) * 2).round() / 2, 8, every)


@MODES
@pytest.mark.parametrize("dtype", list(ref.DTYPES))
def test_extreme_logits(sar, dtype, every):
    d = ref.DTYPES[dtype]
    low, high, inf, nan = torch.finfo(d).min, torch.finfo(d).max, math.inf, math.nan
    rows = [[low] * 6, [high] * 6, [high, low, 0, 1, -1, low], [-inf] * 6, [-inf, -inf, 2, -inf, -inf, 1],
            [low, -inf, low, -inf, -inf, -inf], [nan, 1, 2, 3, nan, 0], [inf, 1, 2, 3, 4, 5], [inf, inf, -inf, 0, 0, 0],
            [-inf, nan, -inf, -inf, -inf, -inf], [0, 0, 0, 0, 0, torch.finfo(d).tiny]]
    check_route(sar, torch.tensor(rows, device="cuda", dtype=d), 4, every)


@MODES
@pytest.mark.parametrize("dtype,bits", [("fp32", [-1, 0x7F800001, -0x7FFFFF, 0x7FFFFFFF]), ("bf16", [-1, 0x7F81, -0x7F, 0x7FFF]),
                                        ("fp16", [-1, 0x7C01, -0x3FF, 0x7FFF])])
def test_every_nan_is_the_greatest(sar, dtype, bits, every):
    """Negative, quiet and signalling ones are equal to each other and above plus infinity."""
    d = ref.DTYPES[dtype]
    for experts in (9, 300):
        x = torch.zeros(1, experts, dtype=d, device="cuda")
        x[0, 1], x[0, 2] = math.inf, -math.inf
        for place, b in zip((3, 4, 6, experts - 1), bits):
            x.view(torch.int32 if d == torch.float32 else torch.int16)[0, place] = b
        assert int(torch.isnan(x).sum()) == 4
        ids, weights = route(sar, x, 6, every)
        assert ids.tolist() == [[3, 4, 6, experts - 1, 1, 0]] and bool(torch.isnan(weights).all())


def backward(sar, dw, x, ids, every, gap=0, inplace=False):
    xv, _ = placed(x, gap)
    out, flat = (xv, None) if inplace else placed(torch.zeros_like(x), gap)
    sar.sar_expert_route_backward(dw, xv, ids, out, softmax=sar.SAR_SOFTMAX_ALL if every else sar.SAR_SOFTMAX_CHOSEN)
    torch.cuda.synchronize()
    if flat is not None:
        assert untouched(out, flat)
    return out


def check_backward(sar, dw, x, ids, every, **kw):
    got = backward(sar, dw, x, ids, every, **kw)
    want, bound = bref.route_backward(dw, x, ids, every)
    ref.check(got, want, ref.rounded(bound, torch.nan_to_num(want), x.dtype), "dlogits")


@MODES
@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("tokens,experts,topk,mask", [
    (1, 1, 1, 0.0), (3, 7, 3, 0.4), (9, 32, 8, 0.0), (32, 128, 8, 0.0), (17, 61, 6, 0.2), (100, 64, 32, 0.1), (13, 65, 16, 0.9),
    (50, 256, 8, 0.0), (7, 257, 12, 0.3), (33, 512, 8, 0.5), (5, 1000, 31, 0.0), (9, 1024, 32, 0.0)])
def test_route_backward(sar, tokens, experts, topk, mask, dtype, every):
    x = scores(tokens, experts, ref.DTYPES[dtype], tokens + experts, mask)
    g = torch.Generator(device="cuda").manual_seed(5)
    dw = torch.randn(tokens, topk, generator=g, device="cuda")
    ids, _ = route(sar, x, topk, every, id_type=torch.int64)
    check_backward(sar, dw, x, ids, every, gap=tokens % 3)
    check_backward(sar, dw.to(x.dtype), x, ids.int(), every, inplace=True)


@MODES
def test_gradient_against_differences(sar, every):
    """Central differences of the 64-bit definition, the choice held fixed: their own error is h^2 / 6 of a third
    derivative (below 1 for a softmax's weights), 1e-8 here, beside the gradient's 1e-6."""
    x = scores(6, 20, torch.float32, 3)
    ids, _ = route(sar, x, 4, every, id_type=torch.int64)
    dw = torch.randn(6, 4, generator=torch.Generator().manual_seed(1)).cuda()
    got = backward(sar, dw, x, ids, every).double()

    def value(z):
        logs = z.gather(1, ids) - torch.logsumexp(z if every else z.gather(1, ids), 1, keepdim=True)
        return (dw.double() * torch.exp(logs)).sum(1)
    h = 1e-4
    for e in range(20):
        step = torch.zeros(6, 20, dtype=torch.float64, device="cuda")
        step[:, e] = h
        slope = (value(x.double() + step) - value(x.double() - step)) / (2 * h)
        assert (got[:, e] - slope).abs().max() < 2e-6


@MODES
def test_ids_given_twice_or_outside_the_experts(sar, every):
    x = scores(5, 9, torch.float32, 4)
    dw = torch.randn(5, 4, generator=torch.Generator().manual_seed(2)).cuda()
    ids = torch.tensor([[3, 3, 3, 1], [0, -1, 9, 0], [-1, -1, -1, -1], [8, 2 ** 31 - 1, -2 ** 31, 8], [5, 4, 5, 4]], device="cuda")
    check_backward(sar, dw, x, ids.int(), every)
    check_backward(sar, dw, x, ids, every)
    far = torch.where((ids < 0) | (ids > 8), 2 ** 32 + 3, ids)            # whose low 32 bits are an expert
    check_backward(sar, dw, x, far, every)
    dropped = dw.clone()
    dropped[(ids < 0) | (ids > 8)] = math.nan                             # never read
    assert torch.equal(backward(sar, dropped, x, ids, every), backward(sar, dw, x, ids, every))


@MODES
def test_route_gradient_of_extreme_logits(sar, every):
    inf, nan = math.inf, math.nan
    x = torch.tensor([[-inf] * 5, [-inf, 1, -inf, 2, -inf], [3e38, -3e38, 3e38, 0, 0], [1, nan, 2, 3, 0], [0, 0, 0, 0, 0]],
                     device="cuda")
    dw = torch.tensor([[1.0, 2.0], [3.0, -1.0], [0.5, 1.0], [1.0, 1.0], [-2.0, 5.0]], device="cuda")
    ids = torch.tensor([[-1, -1], [3, 1], [0, 2], [3, 2], [0, 1]], device="cuda")
    got = backward(sar, dw, x, ids, every)
    assert not got[0].any()
    assert got[1].tolist()[0] == 0.0 and torch.isfinite(got[1]).all()
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[4]).all()
    assert torch.isnan(got[3]).all() if every else torch.isfinite(got[3]).all()


def test_empty_batch_and_refusals(sar):
    x = torch.zeros(0, 8, device="cuda")
    i, w = torch.zeros(0, 2, dtype=torch.int32, device="cuda"), torch.zeros(0, 2, device="cuda")
    sar.sar_expert_route(x, i, w)
    sar.sar_expert_route_backward(w, x, i, x)
    y = torch.zeros(4, 8, device="cuda")
    i, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in (lambda: sar.sar_expert_route(y, i.float(), w), lambda: sar.sar_expert_route(y, i[:3], w),
                lambda: sar.sar_expert_route(y, i, w.half()), lambda: sar.sar_expert_route(y.t(), i, w),
                lambda: sar.sar_expert_route(y, i, w[:, :1]), lambda: sar.sar_expert_route(y.cpu(), i, w),
                lambda: sar.sar_expert_route_backward(w, y, i, y[:3]), lambda: sar.sar_expert_route_backward(w, y, i, y.half())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sar.SarError):
        sar.sar_expert_route(y, torch.zeros(4, 9, dtype=torch.int32, device="cuda"), torch.zeros(4, 9, device="cuda"))
    with pytest.raises(sar.SarError):
        sar.sar_expert_route(y, i, w, softmax=2)


def test_many_tokens_twice_the_same(sar):
    x = scores(40000, 256, torch.bfloat16, 8)
    first = route(sar, x, 8, True)
    again = route(sar, x, 8, True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    best = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(first[0].long(), best.indices[:, :8])


def test_captured_in_a_graph_on_another_stream(sar):
    x = scores(200, 60, torch.float16, 9)
    ids, w = torch.empty(200, 6, dtype=torch.int32, device="cuda"), torch.empty(200, 6, device="cuda")
    dx, dw = torch.empty_like(x), torch.randn(200, 6, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        sar.sar_expert_route(x, ids, w)
        sar.sar_expert_route_backward(dw, x, ids, dx)
    for seed in (10, 11):
        x.copy_(scores(200, 60, torch.float16, seed))
        graph.replay()
        torch.cuda.synchronize()
        want = route(sar, x, 6, False)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
        assert torch.equal(dx, backward(sar, dw, x, ids, False))
