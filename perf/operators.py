"""The operators of a block with layer norm and experts, as they are measured: the cases, their inputs, and each
operator's plain form in elementary torch operations beside the library's calls.

A case is one of

- ``layer_norm``: y = (x - mean) * rstd * weight + bias for each row, with the statistics a backward pass keeps;
- ``layer_norm_backward``: dx, and the gradients of weight and bias, which are sums over the rows;
- ``expert_sort``: a stable counting sort of the (token, choice) slots by expert, with each expert's segment padded to
  ``align`` rows;
- ``expert_dispatch``: each token's row copied to its slots' places, the padding of the segments zeroed;
- ``expert_combine``: the weighted sum of each token's rows (without weights: the gradient of the dispatch);
- ``expert_combine_backward``: the gradients of the rows and of the weights.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
#: The bytes of the largest listed case; a drawn one stays below.
MOST_BYTES = 1.2e9


def listed():
    return [
        # Eight sequences that each decode one token: latency.
        dict(name="norm 8x4096 bf16", op="layer_norm", rows=8, cols=4096, dtype="bf16", wdtype="bf16", bias=True, gap=0),
        # A long batch of a wide model, parameters in 32 bits as mixed-precision training keeps them.
        dict(name="norm 16384x8192 bf16", op="layer_norm", rows=16384, cols=8192, dtype="bf16", wdtype="fp32", bias=True,
             gap=0),
        # One rank's share of a training batch: 64 MiB, the per-rank size of the allreduce's headline.
        dict(name="norm grad 8192x4096 fp16", op="layer_norm_backward", rows=8192, cols=4096, dtype="fp16", wdtype="fp32",
             bias=True, gap=0),
        # Odd sizes in 32 bits: rows that begin at every alignment.
        dict(name="norm grad 4099x1021 fp32", op="layer_norm_backward", rows=4099, cols=1021, dtype="fp32", wdtype="fp32",
             bias=True, gap=0),
        # The routing of 32 decoded tokens, ids as torch.topk gives them.
        dict(name="sort 32x8 of 128", op="expert_sort", tokens=32, topk=8, experts=128, align=1, drop=0.0, wide=True),
        # A training batch's routing, segments padded to a matrix product's tile, some slots dropped.
        dict(name="sort 65536x8 of 256", op="expert_sort", tokens=65536, topk=8, experts=256, align=128, drop=0.02,
             wide=False),
        # 32 decoded tokens to their experts.
        dict(name="dispatch 32x8x2048 bf16", op="expert_dispatch", tokens=32, topk=8, experts=128, align=1, drop=0.0,
             cols=2048, dtype="bf16", gap=0),
        # The rows of a long prompt or training batch: 1 GiB of copies.
        dict(name="dispatch 16384x8x4096 bf16", op="expert_dispatch", tokens=16384, topk=8, experts=256, align=1, drop=0.0,
             cols=4096, dtype="bf16", gap=0),
        # The dispatch's gradient (no weights) of a ragged batch: rows of 3000 bytes, dropped slots, padding.
        dict(name="dispatch grad 1003x6x1500", op="expert_combine", tokens=1003, topk=6, experts=60, align=16, drop=0.1,
             cols=1500, dtype="fp16", weighted=False, wdtype="fp32"),
        # A training batch's rows summed back with the router's weights.
        dict(name="combine 16384x8x4096 bf16", op="expert_combine", tokens=16384, topk=8, experts=256, align=1, drop=0.0,
             cols=4096, dtype="bf16", weighted=True, wdtype="fp32"),
        # A small batch with two choices, in 32 bits.
        dict(name="combine grad 512x2x1024 fp32", op="expert_combine_backward", tokens=512, topk=2, experts=8, align=64,
             drop=0.0, cols=1024, dtype="fp32", wdtype="fp32"),
        # A training batch with wide rows; router weights of the rows' type.
        dict(name="combine grad 8192x4x8192", op="expert_combine_backward", tokens=8192, topk=4, experts=64, align=1,
             drop=0.0, cols=8192, dtype="fp16", wdtype="fp16"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm; one in three is a multiple of 64, if that fits."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    if rng.random() < 1 / 3 and v >= 64:
        v -= v % 64
    return v


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "expert_sort", "expert_dispatch", "expert_combine",
                     "expert_combine_backward"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op.startswith("layer_norm"):
        cols = _spread(rng, 32, 16384)
        most = MOST_BYTES / (3 * SIZE[dtype] * cols)
        return dict(op=op, rows=_spread(rng, 1, int(min(65536, most))), cols=cols, dtype=dtype,
                    wdtype=rng.choice([dtype, "fp32"]), bias=rng.random() < 0.8, gap=rng.choice([0, 0, 0, 24, 64]))
    experts = _spread(rng, 4, 512)
    topk = rng.randint(1, min(8, experts))
    case = dict(op=op, topk=topk, experts=experts, align=rng.choice([1, 1, 16, 128]), drop=rng.choice([0.0, 0.0, 0.05, 0.5]))
    if op == "expert_sort":
        return dict(case, tokens=_spread(rng, 1, 65536), wide=rng.random() < 0.5)
    cols = _spread(rng, 64, 8192)
    case.update(cols=cols, dtype=dtype)
    per_token = (2 * topk + 1) * cols * SIZE[dtype] if op == "expert_combine_backward" else (topk + 1) * cols * SIZE[dtype]
    room = MOST_BYTES - 2 * experts * case["align"] * cols * SIZE[dtype]
    if room < per_token:
        case["align"], room = 1, MOST_BYTES
    case["tokens"] = _spread(rng, 1, max(1, int(min(65536, room / per_token))))
    if op == "expert_dispatch":
        return dict(case, gap=rng.choice([0, 0, 0, 24, 64]))
    case["wdtype"] = rng.choice([dtype, "fp32"])
    if op == "expert_combine":
        case["weighted"] = rng.random() < 0.7
    return case


def _capacity(case):
    """Rows that hold every segment whatever the routing: at most align - 1 more for each expert that gets a token."""
    slots = case["tokens"] * case["topk"]
    return slots + min(case["experts"], slots) * (case["align"] - 1)


def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        n, es, ws = case["rows"] * case["cols"], SIZE[case["dtype"]], SIZE[case["wdtype"]]
        if op == "layer_norm":
            return {"bytes": 2 * n * es + case["cols"] * ws * (2 if case["bias"] else 1) + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * es + 3 * case["cols"] * ws + 8 * case["rows"], "flops": 14 * n}
    tokens, topk, experts = case["tokens"], case["topk"], case["experts"]
    slots = tokens * topk
    if op == "expert_sort":
        return {"bytes": slots * (8 if case["wide"] else 4) + 4 * slots + 4 * _capacity(case) + 8 * experts + 4,
                "flops": 4 * slots}
    kept = slots * (1 - case["drop"])                 # rows that are moved; the mean padding is half of align - 1 a segment
    pad = experts * (case["align"] - 1) / 2 if slots >= experts else 0
    row = case["cols"] * SIZE[case["dtype"]]
    if op == "expert_dispatch":
        return {"bytes": tokens * row + (kept + pad) * row + 4 * slots, "flops": 0}
    if op == "expert_combine":
        w = slots * SIZE[case["wdtype"]] if case["weighted"] else 0
        return {"bytes": kept * row + tokens * row + 4 * slots + w, "flops": 2 * kept * case["cols"]}
    return {"bytes": tokens * row + (2 * kept + pad) * row + 4 * slots + 2 * slots * SIZE[case["wdtype"]],
            "flops": 3 * kept * case["cols"]}


def _matrix(gen, rows, cols, dtype, gap=0, scale=1.0, shift=0.0):
    """Rows of normal values; with a gap, a slice of the columns of a wider matrix."""
    m = torch.randn(rows, cols + gap, generator=gen, device="cuda", dtype=torch.float32)
    m = m.mul_(scale).add_(shift).to(TYPES[dtype])
    return m[:, :cols]


def _routing(gen, case):
    """Ids and weights of each token's choices: popular and unpopular experts, some slots dropped (-1), and with drops
    some tokens (padding of the batch) without any choice."""
    tokens, topk, experts = case["tokens"], case["topk"], case["experts"]
    scores = torch.randn(tokens, experts, generator=gen, device="cuda")
    scores += torch.randn(experts, generator=gen, device="cuda") * 0.7
    best, ids = torch.topk(scores, topk, dim=1)
    weights = torch.softmax(best, dim=1)
    if case["drop"]:
        ids[torch.rand(tokens, topk, generator=gen, device="cuda") < case["drop"]] = -1
        ids[torch.rand(tokens, generator=gen, device="cuda") < 0.02] = -1
    return ids, weights


def _plain_sort(ids, experts, align, capacity):
    flat = ids.reshape(-1).long()
    slots = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(experts + 1, dtype=torch.long, device=key.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts[:experts] + align - 1) // align * align
    offsets = torch.zeros(experts + 1, dtype=torch.long, device=key.device)
    offsets[1:] = torch.cumsum(padded, 0)
    by = key[order]
    place = torch.arange(slots, device=key.device) - (torch.cumsum(counts, 0) - counts)[by] + offsets[by]
    place = torch.where((by < experts) & (place < capacity), place, -1)
    position = torch.empty_like(flat)
    position[order] = place
    source = torch.full((capacity + 1,), -1, dtype=torch.long, device=key.device)
    source[torch.where(place >= 0, place, capacity)] = order
    return counts[:experts].int(), offsets.int(), position.int().view(ids.shape), source[:capacity].int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op.startswith("layer_norm"):
        rows, cols, dtype, wdtype = case["rows"], case["cols"], case["dtype"], case["wdtype"]
        s["x"] = x = _matrix(gen, rows, cols, dtype, case["gap"], 1.5, 0.25)
        s["weight"] = _matrix(gen, 1, cols, wdtype, 0, 0.1, 1.0).view(-1)
        s["mean"], s["rstd"] = (torch.zeros(rows, device="cuda") for _ in range(2))
        if op == "layer_norm":
            s["bias"] = _matrix(gen, 1, cols, wdtype, 0, 0.1).view(-1) if case["bias"] else None
            s["y"] = torch.zeros(rows, cols, dtype=TYPES[dtype], device="cuda")
            return s
        s["mean"] = x.double().mean(1).float()
        s["rstd"] = (x.double().var(1, unbiased=False) + EPS).rsqrt().float()
        s["dy"] = _matrix(gen, rows, cols, dtype, 0, 0.1)
        s["dx"] = torch.zeros(rows, cols, dtype=TYPES[dtype], device="cuda")
        s["dweight"] = torch.zeros(cols, dtype=TYPES[wdtype], device="cuda")
        s["dbias"] = torch.zeros(cols, dtype=TYPES[wdtype], device="cuda") if case["bias"] else None
        return s
    tokens, topk, experts, capacity = case["tokens"], case["topk"], case["experts"], _capacity(case)
    ids, weights = _routing(gen, case)
    s["capacity"] = capacity
    if op == "expert_sort":
        s["ids"] = ids if case["wide"] else ids.int()
        s["counts"] = torch.zeros(experts, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        s["position"] = torch.zeros(tokens, topk, dtype=torch.int32, device="cuda")
        s["source"] = torch.zeros(capacity, dtype=torch.int32, device="cuda")
        return s
    cols, dtype = case["cols"], case["dtype"]
    s["counts"], s["offsets"], s["position"], s["source"] = _plain_sort(ids, experts, case["align"], capacity)
    if op == "expert_dispatch":
        s["x"] = _matrix(gen, tokens, cols, dtype, case["gap"])
        s["rows"] = torch.zeros(capacity, cols, dtype=TYPES[dtype], device="cuda")
        return s
    s["rows"] = _matrix(gen, capacity, cols, dtype)
    s["weights"] = weights.to(TYPES[case["wdtype"]]) if case.get("weighted", True) else None
    if op == "expert_combine":
        s["out"] = torch.zeros(tokens, cols, dtype=TYPES[dtype], device="cuda")
        return s
    s["dout"] = _matrix(gen, tokens, cols, dtype, 0, 0.1)
    s["drows"] = torch.zeros(capacity, cols, dtype=TYPES[dtype], device="cuda")
    s["dweights"] = torch.zeros(tokens, topk, dtype=TYPES[case["wdtype"]], device="cuda")
    return s


def _run_own(s):
    import allreduce_reduction_rank_gb300 as sar
    op = s["op"]
    if op == "layer_norm":
        sar.sar_layer_norm(s["x"], s["y"], s["weight"], s["bias"], s["mean"], s["rstd"], eps=EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "layer_norm_backward":
        if "workspace" not in s:                        # kept by a program for all its calls
            n = sar.sar_layer_norm_backward_workspace_bytes(s["rows"], s["cols"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        sar.sar_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                    workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "expert_sort":
        sar.sar_expert_sort(s["ids"], s["counts"], s["offsets"], s["position"], s["source"], align=s["align"])
        return {"counts": s["counts"], "offsets": s["offsets"], "position": s["position"], "source": s["source"]}
    if op == "expert_dispatch":
        sar.sar_expert_dispatch(s["x"], s["position"], s["rows"], s["counts"], s["offsets"])
        return {"rows": s["rows"]}
    if op == "expert_combine":
        sar.sar_expert_combine(s["rows"], s["position"], s["out"], s["weights"])
        return {"out": s["out"]}
    sar.sar_expert_combine_backward(s["dout"], s["rows"], s["position"], s["weights"], s["drows"], s["dweights"],
                                    s["counts"], s["offsets"])
    return {"drows": s["drows"], "dweights": s["dweights"]}


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "layer_norm":
        x = s["x"].float()
        mean = x.sum(1, keepdim=True) / s["cols"]
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / s["cols"] + EPS)
        y = d * rstd * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean.view(-1), "rstd": rstd.view(-1)}
    if op == "layer_norm_backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        h = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - g.sum(1, keepdim=True) / s["cols"] - h * ((g * h).sum(1, keepdim=True) / s["cols"]))
        wtype = s["weight"].dtype
        return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * h).sum(0).to(wtype),
                "dbias": None if s["dbias"] is None else dy.sum(0).to(wtype)}
    if op == "expert_sort":
        counts, offsets, position, source = _plain_sort(s["ids"], s["experts"], s["align"], s["capacity"])
        return {"counts": counts, "offsets": offsets, "position": position, "source": source}
    if op == "expert_dispatch":
        source = s["source"][:, None]
        return {"rows": torch.where(source >= 0, s["x"][(s["source"].clamp(min=0) // s["topk"]).long()], 0)}
    position = s["position"][:, :, None]
    picked = torch.where(position >= 0, s["rows"][s["position"].clamp(min=0).long()].float(), 0.0)
    if op == "expert_combine":
        if s["weights"] is not None:
            picked = picked * s["weights"].float()[:, :, None]
        return {"out": picked.sum(1).to(s["rows"].dtype)}
    dout = s["dout"].float()
    dweights = (picked * dout[:, None, :]).sum(2).to(s["weights"].dtype)
    slot = s["source"].clamp(min=0).long()
    scaled = dout[slot // s["topk"]] * s["weights"].float().view(-1)[slot][:, None]
    return {"drows": torch.where(s["source"][:, None] >= 0, scaled, 0.0).to(s["rows"].dtype), "dweights": dweights}


def exact(case, seed):
    """The outputs from the definitions in 64 bits. The sort's are whole numbers and have none."""
    op = case["op"]
    if op == "expert_sort":
        return None
    s = prepare(case, seed)
    if op == "layer_norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = (var + EPS).rsqrt()
        y = x.sub_(mean[:, None]).mul_(rstd[:, None]).mul_(s["weight"].double())
        if s["bias"] is not None:
            y.add_(s["bias"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layer_norm_backward":
        # dx as the derivative's three parts: through x, through the mean and through the deviation.
        dy, x, r = s["dy"].double(), s["x"].double(), s["rstd"].double()[:, None]
        h = (x - s["mean"].double()[:, None]).mul_(r)
        dweight, dbias = torch.einsum("rc,rc->c", dy, h), dy.sum(0)
        g = dy.mul_(s["weight"].double())
        along = torch.einsum("rc,rc->r", g, h)[:, None] / s["cols"]
        dx = (g - g.mean(1, keepdim=True)).sub_(h.mul_(along)).mul_(r)
        return {"dx": dx, "dweight": dweight, "dbias": None if s["dbias"] is None else dbias}
    tokens, cols = case["tokens"], case["cols"]
    if op == "expert_dispatch":
        rows = torch.zeros(s["capacity"] + 1, cols, dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):                   # each token's row to its j-th place; dropped ones past the end
            at = s["position"][:, j].long()
            rows[torch.where(at >= 0, at, s["capacity"])] = s["x"].double()
        return {"rows": rows[:-1]}
    weights = torch.ones(tokens, case["topk"], dtype=torch.float64, device="cuda")
    if s["weights"] is not None:
        weights = s["weights"].double()
    if op == "expert_combine":
        out = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):
            at = s["position"][:, j].long()
            kept = torch.nonzero(at >= 0).view(-1)
            out[kept] += s["rows"][at[kept]].double() * weights[kept, j, None]
        return {"out": out}
    drows = torch.zeros(s["capacity"], cols, dtype=torch.float64, device="cuda")
    dweights = torch.zeros(tokens, case["topk"], dtype=torch.float64, device="cuda")
    for j in range(case["topk"]):
        at = s["position"][:, j].long()
        kept = torch.nonzero(at >= 0).view(-1)
        d = s["dout"][kept].double()
        drows[at[kept]] = d * weights[kept, j, None]
        dweights[kept, j] = torch.einsum("tc,tc->t", d, s["rows"][at[kept]].double())
    return {"drows": drows, "dweights": dweights}
