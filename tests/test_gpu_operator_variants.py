"""The variants of the operators' kernels that only larger calls, or calls of
other shapes, reach: both sides of each switch."""
import pytest
import torch

from tests import operator_ref as ref
from tests.test_gpu_experts import MARK, bits, check_combine, check_sort, make, routing, sort
from tests.test_gpu_layer_norm import backward, forward, inputs, placed, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("tokens,topk", [(8191, 1), (8192, 1), (4095, 2), (4096, 2), (2731, 3), (12289, 1)])
@pytest.mark.parametrize("experts", [3, 1024])
def test_sort_around_one_block(sar, tokens, topk, experts):
    """8191 slots are the most of the one block."""
    check_sort(sar, routing(tokens, topk, experts, seed=tokens, drop=0.1), experts, 16)


@pytest.mark.parametrize("capacity", [0, 1, 9000, 17999, 18000, 20000])
def test_sort_of_many_slots_with_too_few_places(sar, capacity):
    check_sort(sar, routing(6000, 3, 40, seed=5), 40, 1, capacity)
    check_sort(sar, routing(6000, 3, 40, seed=5, drop=0.1), 40, 64, capacity)


# More than 608 tokens have other blocks in the dispatch; from 2048 on, other rows go to warps in the gradient.
PLANS = [(608, 4, 9, 1, 0.0), (609, 3, 12, 16, 0.1), (2047, 8, 20, 1, 0.0), (2048, 8, 20, 1, 0.0), (5003, 2, 40, 8, 0.2)]
COLS = [64, 131, 201, 1000, 1025, 1040, 1500, 2040, 2048, 2056]
LAYOUTS = [(0, 0), (8, 0), (5, 3), (0, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "e4m3fn"])
@pytest.mark.parametrize("gap,offset", LAYOUTS)
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_dispatch_of_many_tokens(sar, plan, cols, gap, offset, dtype):
    tokens, topk, experts, align, drop = plan
    counts, offsets, position, src = sort(sar, routing(tokens, topk, experts, seed=1, drop=drop), experts, align)
    td = torch.float8_e4m3fn if dtype == "e4m3fn" else ref.DTYPES[dtype]
    whole = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[torch.empty(0, dtype=td).element_size()]
    x, _ = placed(bits(make(tokens, cols, td)), gap, offset)
    rows, flat = placed(torch.full((src.numel(), cols), 3, dtype=whole, device="cuda"), gap, offset)
    sar.sar_expert_dispatch(x.view(td), position, rows.view(td), counts, offsets)
    torch.cuda.synchronize()
    want = torch.full((src.numel(), cols), 3, dtype=whole, device="cuda")
    want[(torch.arange(src.numel(), device="cuda") < offsets[-1]) & (src < 0)] = 0
    kept = src >= 0
    want[kept] = x[src[kept].long() // topk]
    assert torch.equal(rows, want)
    assert untouched(rows, flat)


@pytest.mark.parametrize("types", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")], ids="/".join)
@pytest.mark.parametrize("cols", COLS + [4080, 4088, 4096])
@pytest.mark.parametrize("plan", PLANS, ids=str)
def test_combine_of_many_tokens(sar, plan, cols, types):
    tokens, topk, experts, align, drop = plan
    dt, wt = (ref.DTYPES[t] for t in types)
    counts, offsets, position, src = sort(sar, routing(tokens, topk, experts, seed=2, drop=drop), experts, align)
    gap, offset = LAYOUTS[(tokens + cols) % len(LAYOUTS)] if cols % 8 else (0, 0)
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


def test_combine_past_32_bits_of_granules(sar):
    """Rows on 2-byte boundaries, of which there are 2^32 elements and more: places no longer fit 32 bits."""
    cols = 4097
    cap = 2 ** 32 // cols + 9
    big = torch.empty(cap, cols, dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[cap - 1, 0], [7, cap - 2], [cap - 3, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    kept = position[position >= 0].long()
    assert big.storage_offset() + (cap - 1) * cols > 2 ** 32 - 2 ** 16
    big[kept] = make(kept.numel(), cols, torch.bfloat16)
    weights = torch.rand(4, 2, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for w in (weights, None):
        out = torch.full((4, cols), MARK, dtype=torch.bfloat16, device="cuda")
        sar.sar_expert_combine(big, position, out, w)
        want = torch.zeros(4, cols, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for j in range(2):
            for t in range(4):
                if int(position[t, j]) >= 0:
                    term = big[int(position[t, j])].double() * (1.0 if w is None else w[t, j].double())
                    want[t] += term
                    size[t] += term.abs()
        ref.check(out, want, ref.rounded(ref.SLACK * 3 * ref.U * size, want, torch.bfloat16), "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("gap,offset", [(0, 0), (5, 3)])
@pytest.mark.parametrize("shape", [(39000, 257), (9740, 1021), (700, 4099), (330, 9001)], ids=str)
def test_in_place_over_many_rows_off_16_bytes(sar, shape, gap, offset, dtype):
    dt = ref.DTYPES[dtype]
    x, dy, w, b = inputs(*shape, dt, torch.float32, seed=4)
    y, mean, rstd = forward(sar, x, w, b, gap=gap, offset=offset)
    z, flat = placed(x, gap, offset)
    sar.sar_layer_norm(z, z, w, b)
    assert torch.equal(z, y) and untouched(z, flat)
    dx, dw, db = backward(sar, dy, x, w, mean, rstd, torch.float32, gap, offset)
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")
    for which in ("dy", "x"):
        (a, fa), (c, fc) = placed(dy, gap, offset), placed(x, gap, offset)
        into, flat = (a, fa) if which == "dy" else (c, fc)
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        sar.sar_layer_norm_backward(a, c, w, mean, rstd, into, dw2, db2, workspace=ws)
        assert torch.equal(into, dx) and torch.equal(dw2, dw) and torch.equal(db2, db) and untouched(into, flat)
