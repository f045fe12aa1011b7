"""Tokens sorted by expert, dispatched and combined, and the gradients, against
one-slot-at-a-time and 64-bit definitions (tests/operator_ref.py)."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_layer_norm import MARK, placed, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def routing(tokens, topk, experts, seed=0, drop=0.0, skew=1.0, wide=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    scores = torch.randn(tokens, experts, generator=g, device="cuda") + skew * torch.randn(experts, generator=g, device="cuda")
    ids = torch.topk(scores, topk, dim=1).indices
    if drop:
        ids[torch.rand(tokens, topk, generator=g, device="cuda") < drop] = -1
        ids[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -1
    return ids if wide else ids.int()


def sort(sar, ids, experts, align=1, capacity=None, source=True):
    tokens, topk = ids.shape
    capacity = sar.sar_expert_rows(tokens, topk, experts, align) if capacity is None else capacity
    bufs = [torch.full((n + 2,), -77, dtype=torch.int32, device="cuda")
            for n in (experts, experts + 1, tokens * topk, capacity)]
    counts, offsets, position, src = (b[1:-1] for b in bufs)
    position = position.view(tokens, topk)
    sar.sar_expert_sort(ids, counts, offsets, position, src if source else None, align=align, capacity=capacity)
    torch.cuda.synchronize()
    assert all(int(b[0]) == -77 and int(b[-1]) == -77 for b in bufs)
    if not source:
        assert bool((src == -77).all())
    return counts, offsets, position, src


def check_sort(sar, ids, experts, align=1, capacity=None):
    counts, offsets, position, src = sort(sar, ids, experts, align, capacity)
    want = ref.expert_sort(ids.tolist(), experts, align, src.numel())
    assert counts.tolist() == want[0]
    assert offsets.tolist() == want[1]
    assert position.tolist() == want[2]
    assert src.tolist() == want[3]
    again = sort(sar, ids, experts, align, capacity, source=False)
    assert all(torch.equal(p, q) for p, q in zip(again[:3], (counts, offsets, position)))


@pytest.mark.parametrize("wide", [True, False], ids=["int64", "int32"])
@pytest.mark.parametrize("tokens,topk,experts,align,drop", [
    (1, 1, 1, 1, 0.0), (1, 2, 3, 1, 0.0), (5, 1, 4, 16, 0.0), (31, 3, 7, 1, 0.2), (32, 8, 128, 1, 0.0),
    (33, 8, 256, 128, 0.0), (257, 4, 64, 8, 0.1), (1000, 6, 60, 1, 0.5), (1021, 5, 1024, 3, 0.0), (4099, 8, 255, 128, 0.05),
    (9001, 2, 1000, 1, 0.0), (20000, 1, 2, 64, 0.3)])
def test_sort(sar, tokens, topk, experts, align, drop, wide):
    check_sort(sar, routing(tokens, topk, experts, seed=tokens, drop=drop, wide=wide), experts, align)


@pytest.mark.parametrize("tokens", [70, 5000])
def test_sort_of_one_sided_routings(sar, tokens):
    """Every slot to one expert; the same expert twice for a token; nothing kept."""
    for e in (0, 6):
        check_sort(sar, torch.full((tokens, 3), e, device="cuda"), 7, 16)
    check_sort(sar, torch.full((tokens, 2), -1, device="cuda"), 5, 4)
    check_sort(sar, torch.arange(tokens * 2, device="cuda").view(tokens, 2) % 9, 9, 1)
    check_sort(sar, (torch.arange(tokens * 2, device="cuda").view(tokens, 2) // 7) % 9, 9, 2)


def test_sort_drops_ids_outside_the_experts(sar):
    """Ids far outside, whose low 32 bits would be an expert, are dropped too."""
    ids = torch.tensor([[0, 2 ** 32], [3, -1], [2 ** 40 + 1, 1], [-2 ** 63, 2 ** 63 - 1], [2, 4]], device="cuda")
    check_sort(sar, ids, 4, 1)
    assert sort(sar, ids, 4)[2].tolist() == [[0, -1], [3, -1], [-1, 1], [-1, -1], [2, -1]]


@pytest.mark.parametrize("capacity", [0, 1, 100, 511, 512, 600])
def test_sort_with_too_few_places(sar, capacity):
    check_sort(sar, routing(256, 2, 8, seed=3), 8, 1, capacity)
    check_sort(sar, routing(256, 2, 8, seed=4), 8, 64, capacity)


def test_sort_of_an_empty_batch(sar):
    counts, offsets, position, src = sort(sar, torch.empty(0, 4, dtype=torch.int64, device="cuda"), 6, 8, 10)
    assert counts.tolist() == [0] * 6 and offsets.tolist() == [0] * 7 and src.tolist() == [-1] * 10


def test_sort_of_many_slots(sar):
    """A million slots against torch's stable sort."""
    tokens, topk, experts, align = 131072, 8, 300, 128
    ids = routing(tokens, topk, experts, seed=6, drop=0.01)
    counts, offsets, position, src = sort(sar, ids, experts, align)
    flat = torch.where(ids < 0, experts, ids).view(-1)
    key, order = torch.sort(flat, stable=True)
    c = torch.bincount(flat, minlength=experts + 1)
    assert torch.equal(counts.long(), c[:experts])
    o = torch.cat([c.new_zeros(1), torch.cumsum((c[:experts] + align - 1) // align * align, 0)])
    assert torch.equal(offsets.long(), o)
    place = torch.arange(flat.numel(), device="cuda") - (torch.cumsum(c, 0) - c)[key] + o[key.clamp(max=experts - 1)]
    want = torch.empty_like(flat)
    want[order] = torch.where(key < experts, place, -1)
    assert torch.equal(position.view(-1).long(), want)
    at = torch.full((src.numel(),), -1, dtype=torch.long, device="cuda")
    at[want[want >= 0]] = torch.nonzero(want >= 0).view(-1)
    assert torch.equal(src.long(), at)


def make(tokens, cols, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype == torch.uint8:
        return torch.randint(0, 256, (tokens, cols), generator=g, dtype=torch.uint8, device="cuda")
    if dtype == torch.float8_e4m3fn:
        return make(tokens, cols, torch.uint8, seed).view(dtype)
    return torch.randn(tokens, cols, generator=g, device="cuda").to(dtype)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


PLANS = [(1, 1, 1, 1, 0.0), (3, 2, 4, 1, 0.0), (40, 8, 16, 1, 0.0), (101, 3, 12, 16, 0.3), (64, 9, 20, 8, 0.1),
         (300, 17, 40, 4, 0.0), (7, 2, 100, 128, 0.0)]
COLS = [1, 7, 64, 100, 257, 1024, 1500, 4096, 9000]
LAYOUTS = [(0, 0), (8, 0), (0, 1), (5, 3), (16, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "e4m3fn", "e4m3b15"])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_dispatch(sar, plan, cols, dtype):
    tokens, topk, experts, align, drop = plan
    td = {"e4m3fn": torch.float8_e4m3fn, "e4m3b15": torch.uint8}.get(dtype) or ref.DTYPES[dtype]
    counts, offsets, position, src = sort(sar, routing(tokens, topk, experts, seed=1, drop=drop), experts, align)
    x = make(tokens, cols, td)
    gap, offset = LAYOUTS[(tokens + cols) % len(LAYOUTS)]
    for clear in (True, False):
        if x.element_size() == 1:                       # marks and copies in plain bytes
            flat = torch.full((offset + src.numel() * (cols + gap) + 64,), 3, dtype=torch.uint8, device="cuda")
            rows = flat[offset:offset + src.numel() * (cols + gap)].view(-1, cols + gap)[:, :cols]
            rows, flat = rows.view(td), flat
        else:
            rows, flat = placed(torch.full((src.numel(), cols), MARK, dtype=td, device="cuda"), gap, offset)
        sar.sar_expert_dispatch(x, position, rows, counts if clear else None, offsets if clear else None,
                                dtype=sar.SAR_FP8_E4M3B15 if dtype == "e4m3b15" else None)
        torch.cuda.synchronize()
        want = torch.full_like(bits(rows), 3) if x.element_size() == 1 else bits(torch.full_like(rows, MARK))
        if clear:
            inside = (torch.arange(src.numel(), device="cuda") < offsets[-1]) & (src < 0)
            want[inside] = 0
        kept = src >= 0
        want[kept] = bits(x)[src[kept].long() // topk]
        assert torch.equal(bits(rows), want)
        if x.element_size() == 1:
            rest = flat.clone()
            rest[offset:offset + src.numel() * (cols + gap)].view(-1, cols + gap)[:, :cols] = 3
            assert bool((rest == 3).all())
        else:
            assert untouched(rows, flat)


def check_combine(sar, rows, position, weights, gap=0, offset=0):
    out, flat = placed(torch.full((position.shape[0], rows.shape[1]), MARK, dtype=rows.dtype, device="cuda"), gap, offset)
    sar.sar_expert_combine(rows, position, out, weights)
    torch.cuda.synchronize()
    want, bound = ref.combine(rows, position, weights)
    ref.check(out, want, ref.rounded(bound, want, rows.dtype), "out")
    assert untouched(out, flat)
    return out


TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_combine_and_its_gradient(sar, plan, cols, types):
    tokens, topk, experts, align, drop = plan
    dt, wt = (ref.DTYPES[t] for t in types)
    counts, offsets, position, src = sort(sar, routing(tokens, topk, experts, seed=2, drop=drop), experts, align)
    gap, offset = LAYOUTS[(tokens + cols) % len(LAYOUTS)]
    rows, _ = placed(make(src.numel(), cols, dt, seed=3), gap, offset)
    weights = torch.rand(tokens, topk, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(wt)
    check_combine(sar, rows, position, weights, gap, offset)
    check_combine(sar, rows, position, None, gap, offset)

    dout, _ = placed(make(tokens, cols, dt, seed=5), gap, offset)
    drows, flat = placed(torch.full((src.numel(), cols), MARK, dtype=dt, device="cuda"), gap, offset)
    dweights = torch.full((tokens, topk), MARK, dtype=wt, device="cuda")
    sar.sar_expert_combine_backward(dout, rows, position, weights, drows, dweights, counts, offsets)
    torch.cuda.synchronize()
    (wr, ww), (br, bw) = ref.combine_backward(dout, rows, position, weights, src.numel())
    total = int(offsets[-1])
    ref.check(drows[:total], wr[:total], ref.rounded(br, wr, dt)[:total], "drows")
    assert bool((drows[total:] == MARK).all()) and untouched(drows, flat)
    ref.check(dweights, ww, ref.rounded(bw, ww, wt), "dweights")

    alone, flat = placed(torch.full((src.numel(), cols), MARK, dtype=dt, device="cuda"), gap, offset)
    sar.sar_expert_combine_backward(dout, None, position, weights, alone)         # no padding cleared, no dweights
    torch.cuda.synchronize()
    kept = src >= 0
    assert torch.equal(alone[kept], drows[kept]) and bool((alone[~kept] == MARK).all()) and untouched(alone, flat)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cols", [9, 1024])
def test_dropped_slots_are_not_read(sar, cols, dtype):
    """NaN in the weights of dropped slots and in rows that no slot has reaches nothing; a token without a kept slot
    gets zeros, and zero gradients."""
    dt = ref.DTYPES[dtype]
    position = torch.tensor([[2, -1, 0], [-1, -1, -1], [3, 5, -1], [99, 6, -7]], dtype=torch.int32, device="cuda")
    rows = make(8, cols, dt)
    rows[[1, 4, 7]] = float("nan")
    weights = torch.rand(4, 3, device="cuda") + 0.5
    weights[position < 0] = float("nan")
    weights[3, 0] = float("inf")                         # place 99 does not exist
    out = check_combine(sar, rows, torch.where(position > 7, -1, position), weights)
    got = torch.empty_like(out)
    sar.sar_expert_combine(rows, position, got, weights)
    assert torch.equal(got, out) and bool((out[1] == 0).all())
    dout, drows, dw = make(4, cols, dt, 1), torch.full((8, cols), MARK, dtype=dt, device="cuda"), torch.empty(4, 3, device="cuda")
    sar.sar_expert_combine_backward(dout, rows, position, weights, drows, dw)
    assert bool(torch.isfinite(dw).all()) and bool((dw[1] == 0).all()) and float(dw[3, 0]) == 0 and float(dw[3, 2]) == 0
    assert bool((drows[[1, 4, 7]] == MARK).all()) and bool(torch.isfinite(drows).all())


@pytest.mark.parametrize("cols", [5, 64, 1024])
def test_special_values_of_kept_slots(sar, cols):
    """Infinities and NaN of kept rows come through; one kept row without weights is the identity, -0 included."""
    rows = make(6, cols, torch.float16)
    rows[1, 0], rows[2, cols - 1], rows[3] = float("inf"), float("nan"), -0.0
    position = torch.tensor([[0, 1], [2, 4], [3, -1], [-1, 5]], dtype=torch.int32, device="cuda")
    out = torch.empty(4, cols, dtype=torch.float16, device="cuda")
    sar.sar_expert_combine(rows, position, out)
    assert float(out[0, 0]) == float("inf") and bool(torch.isnan(out[1, cols - 1]))
    assert torch.equal(bits(out[2]), bits(rows[3])) and torch.equal(bits(out[3]), bits(rows[5]))


def test_the_same_place_for_every_token(sar):
    """The gradient of the dispatch sums over a token's choices; one row read by many tokens is fine too."""
    rows = make(3, 512, torch.bfloat16)
    check_combine(sar, rows, torch.ones(500, 4, dtype=torch.int32, device="cuda"), None)


@pytest.mark.parametrize("cols", [48, 1000])
def test_gradients_against_differences(sar, cols):
    """The combine is linear in its rows and in its weights, so a difference of two calls is its derivative up to the
    rounding of the two."""
    counts, offsets, position, src = sort(sar, routing(30, 3, 8, seed=7, drop=0.2), 8, 4)
    rows, dout = make(src.numel(), cols, torch.float32, 1), make(30, cols, torch.float32, 2)
    weights, along_w, along_r = torch.rand(30, 3, device="cuda"), torch.randn(30, 3, device="cuda"), make(src.numel(), cols, torch.float32, 3)
    drows, dw = torch.zeros_like(rows), torch.zeros_like(weights)
    sar.sar_expert_combine_backward(dout, rows, position, weights, drows, dw, counts, offsets)
    (er, ew), (br, bw) = ref.combine_backward(dout, rows, position, weights, src.numel())
    for r, w, grad, along, bound in ((along_r, 0, drows, along_r, br + ref.U * er.abs()), (0, along_w, dw, along_w, bw + ref.U * ew.abs())):
        ends, room = [], 0.0
        for sign in (1, -1):
            out = torch.empty(30, cols, device="cuda")
            moved_r, moved_w = rows + sign * 0.5 * r, weights + sign * 0.5 * w
            sar.sar_expert_combine(moved_r, position, out, moved_w)
            want, b = ref.combine(moved_r, position, moved_w)
            # the moved inputs are rounded themselves: one more unit of their magnitude
            room += ((ref.rounded(b, want, torch.float32) + 2 * b) * dout.double().abs()).sum().item()
            ends.append((out.double() * dout.double()).sum().item())
        live = (src >= 0)[:, None] if r is along_r else torch.ones_like(along, dtype=torch.bool)
        own = (grad.double() * along.double() * live).sum().item()
        allowed = room + (bound * along.double().abs() * live).sum().item()
        assert abs(ends[0] - ends[1] - own) <= allowed, (ends, own, allowed)
        assert allowed < 0.01 * (grad.double() * along.double()).abs().sum().item()


def test_dispatch_and_combine_are_each_other_s_adjoint(sar):
    """<dispatch(x), r> = <x, combine(r)> for whole numbers, exactly."""
    counts, offsets, position, src = sort(sar, routing(200, 4, 16, seed=8, drop=0.1), 16, 8)
    x = torch.randint(-8, 9, (200, 256), device="cuda").float()
    r = torch.randint(-8, 9, (src.numel(), 256), device="cuda").float()
    rows, back = torch.zeros_like(r), torch.empty_like(x)
    sar.sar_expert_dispatch(x, position, rows, counts, offsets)
    sar.sar_expert_combine(r, position, back)
    assert (rows.double() * r.double()).sum().item() == (x.double() * back.double()).sum().item()


def test_in_place_gradient_of_the_rows(sar):
    counts, offsets, position, src = sort(sar, routing(50, 2, 6, seed=9), 6, 8)
    for cols in (40, 1024, 3001):
        rows, dout = make(src.numel(), cols, torch.bfloat16, 1), make(50, cols, torch.bfloat16, 2)
        weights = torch.rand(50, 2, device="cuda")
        apart, dw, dw2 = torch.zeros_like(rows), torch.zeros_like(weights), torch.zeros_like(weights)
        sar.sar_expert_combine_backward(dout, rows, position, weights, apart, dw, counts, offsets)
        sar.sar_expert_combine_backward(dout, rows, position, weights, rows, dw2, counts, offsets)
        total = int(offsets[-1])
        assert torch.equal(rows[:total], apart[:total]) and torch.equal(dw, dw2)


def test_nothing_to_do(sar):
    empty = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    rows = torch.full((4, 16), MARK, device="cuda")
    none = torch.empty(0, 16, device="cuda")
    sar.sar_expert_dispatch(none, empty, rows)
    sar.sar_expert_combine(rows, empty, none)
    sar.sar_expert_combine_backward(none, rows, empty, torch.empty(0, 2, device="cuda"), rows, torch.empty(0, 2, device="cuda"))
    assert bool((rows == MARK).all())
    # no place at all: every slot is dropped
    position = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    out, dw = torch.full((3, 16), MARK, device="cuda"), torch.full((3, 2), MARK, device="cuda")
    sar.sar_expert_dispatch(torch.ones(3, 16, device="cuda"), position, none)
    sar.sar_expert_combine(none, position, out)
    sar.sar_expert_combine_backward(out, none, position, torch.ones(3, 2, device="cuda"), none, dw)
    assert bool((out == 0).all()) and bool((dw == 0).all())
    # no columns
    sar.sar_expert_combine_backward(torch.empty(3, 0, device="cuda"), torch.empty(2, 0, device="cuda"), position,
                                    torch.ones(3, 2, device="cuda"), torch.empty(2, 0, device="cuda"), dw.fill_(MARK))
    assert bool((dw == 0).all())


def test_captured_in_a_graph_and_on_another_stream(sar):
    tokens, topk, experts, cols = 100, 4, 16, 512
    ids = routing(tokens, topk, experts, seed=10)
    cap = sar.sar_expert_rows(tokens, topk, experts, 8)
    counts, offsets, src = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (experts, experts + 1, cap))
    position = torch.zeros(tokens, topk, dtype=torch.int32, device="cuda")
    x, rows, out = make(tokens, cols, torch.bfloat16), torch.zeros(cap, cols, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    weights, drows, dw = torch.rand(tokens, topk, device="cuda"), torch.zeros_like(rows), torch.zeros(tokens, topk, device="cuda")

    def step():
        sar.sar_expert_sort(ids, counts, offsets, position, src, align=8)
        sar.sar_expert_dispatch(x, position, rows, counts, offsets)
        sar.sar_expert_combine(rows, position, out, weights)
        sar.sar_expert_combine_backward(x, rows, position, weights, drows, dw, counts, offsets)
        return [t.clone() for t in (counts, offsets, position, src, rows, out, drows, dw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    ids.copy_(routing(tokens, topk, experts, seed=11, drop=0.2))
    rows.zero_(), drows.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in got]
    rows.zero_(), drows.zero_()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_offsets_past_32_bits(sar):
    """Rows whose elements lie past 2^31 from the first."""
    cols = 4096
    cap = 2 ** 31 // cols + 9
    big = torch.empty(cap, cols, dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[cap - 1, 0], [cap - 2, 5]], dtype=torch.int32, device="cuda")
    x = make(2, cols, torch.bfloat16)
    sar.sar_expert_dispatch(x, position, big)
    for t in range(2):
        for j in range(2):
            assert torch.equal(big[position[t, j]], x[t])
    out = torch.empty_like(x)
    sar.sar_expert_combine(big, position, out)
    assert torch.equal(out, (x.float() * 2).bfloat16())
    weights, dw = torch.tensor([[0.5, 2.0], [1.0, 0.25]], device="cuda"), torch.empty(2, 2, device="cuda")
    sar.sar_expert_combine_backward(x, big, position, weights, big, dw)
    want = (x.double() ** 2).sum(1)
    assert torch.allclose(dw.double(), want[:, None].expand(2, 2), rtol=ref.SLACK * ref.row_depth(cols) * ref.U)
    assert torch.equal(big[cap - 2], x[1]) and torch.equal(big[0], (x[0].float() * 2).bfloat16())
