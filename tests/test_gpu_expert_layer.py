"""The expert layer of a few tokens (sar_expert_layer) against its 64-bit
definition (tests/block_ref.py), and against the way of long batches: sort,
dispatch, a product for each segment, combine."""
import math

import pytest
import torch

from tests import block_ref as bref
from tests import operator_ref as ref
from tests.test_gpu_layer_norm import placed, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def case(tokens, topk, experts, cols, hidden, dtype, gated=True, drop=0.0, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = ref.DTYPES[dtype]
    x = (scale * torch.randn(tokens, cols, generator=g, device="cuda")).to(d)
    w_in = (torch.randn(experts, (2 if gated else 1) * hidden, cols, generator=g, device="cuda") / max(1, cols) ** 0.5).to(d)
    w_out = (torch.randn(experts, cols, hidden, generator=g, device="cuda") / max(1, hidden) ** 0.5).to(d)
    ids = torch.rand(tokens, experts, generator=g, device="cuda").argsort(1)[:, :topk].contiguous()
    if drop:
        ids[torch.rand(tokens, topk, generator=g, device="cuda") < drop] = -1
        ids[-1] = -1
    weights = torch.rand(tokens, topk, generator=g, device="cuda")
    return x, ids, w_in, w_out, weights


def act_code(sar, act):
    return {"silu": sar.SAR_ACT_SILU, "gelu": sar.SAR_ACT_GELU, "relu": sar.SAR_ACT_RELU}[act]


def layer(sar, x, ids, w_in, w_out, weights, act="silu", gap=0, offset=0, out=None):
    xv, _ = placed(x, gap, offset)
    ov, flat = placed(torch.zeros_like(x), gap, offset)
    need = sar.sar_expert_layer_workspace_bytes(x.shape[0], ids.shape[1], w_in.shape[0], x.shape[1], w_out.shape[2])
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")           # NaN all over
    sar.sar_expert_layer(xv, ids, w_in, w_out, ov, weights, activation=act_code(sar, act), workspace=ws[:need])
    torch.cuda.synchronize()
    assert untouched(ov, flat) and bool((ws[need:] == 0xFF).all())
    return ov


def check_layer(sar, x, ids, w_in, w_out, weights, act="silu", gated=True, **kw):
    got = layer(sar, x, ids, w_in, w_out, weights, act, **kw)
    want, bound = bref.expert_layer(x, ids, w_in, w_out, weights, gated, act)
    ref.check(got, want, ref.rounded(bound, want, x.dtype), "out")
    return got


SIZES = [(1, 1, 1, 1, 1), (1, 2, 3, 8, 16), (1, 8, 16, 256, 96), (2, 1, 1, 64, 32), (3, 2, 5, 40, 24), (9, 1, 1, 128, 64),
         (5, 3, 7, 33, 17), (17, 3, 20, 101, 55), (8, 8, 8, 72, 200), (33, 1, 2, 136, 40), (40, 2, 2, 64, 72),
         (64, 4, 16, 96, 64), (70, 1, 1, 48, 56), (1, 4, 1024, 16, 8), (2, 2, 4, 2048, 24), (2, 2, 4, 24, 2048),
         (3, 1, 2, 1000, 520), (16, 2, 4, 16, 1), (4, 2, 4, 1, 64), (1, 32, 40, 64, 64)]


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "gelu"), (True, "gelu"), (False, "relu")])
@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", SIZES)
def test_layer(sar, tokens, topk, experts, cols, hidden, gated, act, dtype):
    if act == "gelu" and gated and tokens > 9:
        pytest.skip("the pairing is covered by the small ones")
    x, ids, w_in, w_out, weights = case(tokens, topk, experts, cols, hidden, dtype, gated, seed=tokens + cols)
    check_layer(sar, x, ids, w_in, w_out, weights, act, gated)
    check_layer(sar, x, ids.int(), w_in, w_out, weights.to(x.dtype), act, gated, gap=3, offset=1)


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", [(6, 3, 9, 64, 48), (40, 4, 8, 136, 72), (20, 2, 30, 65, 31)])
def test_dropped_choices(sar, tokens, topk, experts, cols, hidden, dtype):
    x, ids, w_in, w_out, weights = case(tokens, topk, experts, cols, hidden, dtype, drop=0.3, seed=7)
    weights[ids < 0] = math.nan                                                   # never read
    got = check_layer(sar, x, ids, w_in, w_out, weights)
    assert not got[-1].any()
    far = torch.where(ids < 0, 2 ** 32 + 1, ids)                                  # whose low 32 bits are an expert
    assert torch.equal(layer(sar, x, far, w_in, w_out, weights), got)
    assert torch.equal(layer(sar, x, torch.where(ids < 0, experts, ids).int(), w_in, w_out, weights), got)
    assert not layer(sar, x, torch.full_like(ids, -1), w_in, w_out, weights).any()


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
def test_one_expert_for_all_and_the_same_twice(sar, dtype):
    x, ids, w_in, w_out, weights = case(100, 3, 6, 80, 56, dtype, seed=8)
    for e in (0, 5):
        check_layer(sar, x, torch.full_like(ids, e), w_in, w_out, weights)
    ids[:, 1] = ids[:, 0]
    check_layer(sar, x, ids, w_in, w_out, None)


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
def test_the_most_slots(sar, dtype):
    x, ids, w_in, w_out, weights = case(128, 8, 30, 64, 40, dtype, seed=9)
    check_layer(sar, x, ids, w_in, w_out, weights)


def test_values_past_the_range_of_16_bits(sar):
    """h reaches 2^20 and more, past binary16's largest value; the output does not."""
    x, ids, w_in, w_out, weights = case(5, 2, 4, 64, 48, "fp16", seed=10, scale=2000.0)
    check_layer(sar, x, ids, w_in, (w_out.float() * 2.0 ** -12).half(), weights)
    x, ids, w_in, w_out, weights = case(5, 2, 4, 64, 48, "fp16", seed=11, scale=2.0 ** -9)
    check_layer(sar, x, ids, w_in, w_out * 64, weights)                          # h of 2^-20


def test_long_sums_in_binary32_stay_exact(sar):
    """Additions rounded to nearest err independently: over 4096 of k, 64 of them a warp, by sqrt(64) * 2^-24 / sqrt(3) of
    the sum in the mean; the tensor cores' sums of 16 of k, cut off, by up to 4 * 2^-24 of themselves.  Both products:
    1.1e-6.  A chain of cut-off sums over all of k errs by 1e-5."""
    x, ids, w_in, w_out, weights = case(6, 2, 4, 4096, 4096, "fp32", seed=20)
    got = layer(sar, x, ids, w_in, w_out, weights).double()
    want, _ = bref.expert_layer(x, ids, w_in, w_out, weights, True, "silu")
    assert (got - want).norm() / want.norm() < 1.1e-6


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
def test_infinities_and_nan_stay_with_their_token(sar, dtype):
    x, ids, w_in, w_out, weights = case(12, 2, 5, 64, 48, dtype, seed=12)
    clean = layer(sar, x, ids, w_in, w_out, weights)
    x[3, 5], x[7, 0] = math.nan, math.inf
    got = layer(sar, x, ids, w_in, w_out, weights)
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[7]).any()
    rest = [t for t in range(12) if t not in (3, 7)]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("tokens", [0, 3])
def test_nothing_inside(sar, tokens):
    x, ids, w_in, w_out, weights = case(tokens, 2, 4, 16, 0, "bf16", seed=1)
    out = torch.ones(tokens, 16, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sar.sar_expert_layer_workspace_bytes(tokens, 2, 4, 16, 0), dtype=torch.uint8, device="cuda")
    sar.sar_expert_layer(x, ids, w_in, w_out, out, weights, workspace=ws)
    assert not out.any()


@pytest.mark.parametrize("dtype,unit", [("bf16", 2.0 ** -8), ("fp16", 2.0 ** -11)])
def test_as_the_way_of_long_batches(sar, dtype, unit):
    """Router, then the layer; or the router, sort, dispatch, products and combine: the second rounds z, h, the rows and
    the sum to the type, each by up to half a unit, the first only the sum; 8 units bound the mean."""
    tokens, topk, experts, cols, hidden = 24, 3, 8, 128, 64
    x, _, w_in, w_out, _ = case(tokens, topk, experts, cols, hidden, dtype, seed=13)
    logits = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(3)).cuda()
    ids, weights = torch.empty(tokens, topk, dtype=torch.int32, device="cuda"), torch.empty(tokens, topk, device="cuda")
    sar.sar_expert_route(logits, ids, weights)
    got = layer(sar, x, ids, w_in, w_out, weights)
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1))
    position = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
    sar.sar_expert_sort(ids, counts, offsets, position, align=8)
    rows = torch.empty(sar.sar_expert_rows(tokens, topk, experts, 8), cols, dtype=x.dtype, device="cuda")
    made, out = torch.zeros_like(rows), torch.empty_like(x)
    sar.sar_expert_dispatch(x, position, rows, counts, offsets)
    for e, (a, b) in enumerate(zip(offsets.tolist(), offsets.tolist()[1:])):
        z = rows[a:b] @ w_in[e].T
        made[a:b] = (torch.nn.functional.silu(z[:, :hidden]) * z[:, hidden:]) @ w_out[e].T
    sar.sar_expert_combine(made, position, out, weights)
    assert (got.double() - out.double()).norm() / out.double().norm() < 8 * unit


def test_captured_twice_over_one_workspace(sar):
    a = case(6, 2, 8, 128, 96, "bf16", seed=14)
    b = case(3, 4, 8, 64, 200, "fp16", seed=15)
    need = max(sar.sar_expert_layer_workspace_bytes(c[0].shape[0], c[1].shape[1], 8, c[0].shape[1], c[3].shape[2]) for c in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(c[0]) for c in (a, b)], []
    for c, out in zip((a, b), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sar.sar_expert_layer(c[0], c[1], c[2], c[3], out, c[4], workspace=ws)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, out in zip((a, b), outs):
        assert torch.equal(out, layer(sar, *c))


def test_calls_at_once(sar):
    cs = [case(1, 8, 32, 256, 96, "bf16", seed=16), case(1, 1, 1, 64, 40, "fp16", seed=17), case(40, 4, 8, 136, 72, "bf16", seed=18),
          case(3, 2, 5, 33, 17, "fp32", seed=19)]
    want = [layer(sar, *c) for c in cs]
    outs = [torch.empty_like(c[0]) for c in cs]
    spaces = [torch.empty(sar.sar_expert_layer_workspace_bytes(c[0].shape[0], c[1].shape[1], c[2].shape[0], c[0].shape[1], c[3].shape[2]),
                          dtype=torch.uint8, device="cuda") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (x, ids, w_in, w_out, weights), out, ws, s in zip(cs, outs, spaces, streams):
            sar.sar_expert_layer(x, ids, w_in, w_out, out, weights, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_refusals(sar):
    x, ids, w_in, w_out, weights = case(4, 2, 3, 16, 8, "bf16")
    out = torch.empty_like(x)
    ws = torch.empty(sar.sar_expert_layer_workspace_bytes(4, 2, 3, 16, 8), dtype=torch.uint8, device="cuda")

    def call(x=x, ids=ids, w_in=w_in, w_out=w_out, out=out, weights=weights, ws=ws, **kw):
        sar.sar_expert_layer(x, ids, w_in, w_out, out, weights, workspace=ws, **kw)
    call()
    for kw in (dict(x=x.float()), dict(w_in=w_in[:, :15]), dict(w_in=w_in[:2]), dict(w_out=w_out.transpose(1, 2)),
               dict(out=out[:3]), dict(ids=ids[:3]), dict(ids=ids.float()), dict(weights=weights.double()),
               dict(weights=weights[:, :1]), dict(w_in=w_in.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(ws=None), dict(ws=ws[:-1]), dict(activation=3), dict(ws=ws[1:])):
        with pytest.raises(sar.SarError):
            call(**kw)
