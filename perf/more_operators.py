"""The operators that a block with experts needs beside those of perf/operators.py, as they are measured: the cases, their
inputs, and each operator's plain form in elementary torch operations beside the library's calls.

A case is one of

- ``route``: each token's best ``topk`` of its experts' logits and their softmax, over the chosen ones or over all;
- ``route_backward``: the logits' gradient from that of the weights;
- ``layer``: the whole expert layer of a few tokens that are being decoded, out = sum of weight * w_out . act(w_in . x);
- ``orthogonalize``: a gradient's (or a batch of them) Newton-Schulz iteration towards the nearest orthogonal matrix, what
  is applied as the update of a matrix after its gradient has been summed over the ranks.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS, EPS = 5, 1e-7
#: The bytes of weights of the largest listed layer, the bytes of the largest listed routing and the operations of the
#: largest listed orthogonalisation; a drawn case stays below.
MOST_WEIGHTS, MOST_ROUTING, MOST_FLOPS = 1.7e9, 7.4e7, 2.0e12


def listed():
    return [
        # 32 decoded tokens' router, logits in 32 bits: latency.
        dict(name="route 32x128 top 8", op="route", tokens=32, experts=128, topk=8, dtype="fp32", wdtype="fp32", every=False,
             wide=False, mask=0.0),
        # A training batch's router; softmax over all experts; ids as torch.topk gives them.
        dict(name="route 65536x256 top 8", op="route", tokens=65536, experts=256, topk=8, dtype="fp32", wdtype="fp32",
             every=True, wide=True, mask=0.0),
        # A ragged batch with masked experts and padding tokens, whose rows have nothing to choose.
        dict(name="route grad 1003x60 top 6", op="route_backward", tokens=1003, experts=60, topk=6, dtype="fp16",
             wdtype="fp32", every=False, wide=False, mask=0.2),
        # A training batch's gradient through the softmax over all experts.
        dict(name="route grad 65536x256 top 8", op="route_backward", tokens=65536, experts=256, topk=8, dtype="fp32",
             wdtype="fp32", every=True, wide=True, mask=0.0),
        # One decoded token: the weights of its eight experts are read once.
        dict(name="layer 1x8 of 128, 2048/768", op="layer", tokens=1, topk=8, experts=128, cols=2048, hidden=768,
             dtype="bf16", wdtype="fp32", gated=True, act="silu", drop=0.0),
        # 32 decoded tokens, which between them take nearly every expert.
        dict(name="layer 32x8 of 128, 2048/768", op="layer", tokens=32, topk=8, experts=128, cols=2048, hidden=768,
             dtype="bf16", wdtype="fp32", gated=True, act="silu", drop=0.0),
        # 64 tokens and few, large experts: 16 tokens for each.
        dict(name="layer 64x2 of 8, 4096/8192", op="layer", tokens=64, topk=2, experts=8, cols=4096, hidden=8192,
             dtype="fp16", wdtype="fp16", gated=True, act="silu", drop=0.0),
        # Odd sizes in 32 bits without a gate, some choices dropped: rows that begin at every alignment.
        dict(name="layer 17x3 of 20, 1021/515", op="layer", tokens=17, topk=3, experts=20, cols=1021, hidden=515,
             dtype="fp32", wdtype="fp32", gated=False, act="gelu", drop=0.1),
        # Small matrices, a batch of them: latency of a chain of fifteen products.
        dict(name="orthogonal 8x128x128 fp32", op="orthogonalize", batch=8, rows=128, cols=128, dtype="fp32", gap=0),
        # A tall ragged matrix in 16 bits, a slice of the columns of a wider one.
        dict(name="orthogonal 2x1003x357 fp16", op="orthogonalize", batch=2, rows=1003, cols=357, dtype="fp16", gap=24),
        # The experts' gradients of block_step's default sizes.
        dict(name="orthogonal 16x1024x1024 fp32", op="orthogonalize", batch=16, rows=1024, cols=1024, dtype="fp32", gap=0),
        # One large projection's gradient.
        dict(name="orthogonal 4096x4096 bf16", op="orthogonalize", batch=1, rows=4096, cols=4096, dtype="bf16", gap=0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm; one in three is a multiple of 64, if that fits."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = min(high, max(low, v))
    if rng.random() < 1 / 3 and v >= 64:
        v -= v % 64
    return v


def draw(rng):
    op = rng.choice(["route", "route_backward", "layer", "layer", "orthogonalize", "orthogonalize"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op.startswith("route"):
        experts = _spread(rng, 4, 1024)
        most = MOST_ROUTING / (experts * SIZE[dtype] + 96)
        return dict(op=op, tokens=_spread(rng, 1, int(min(65536, most))), experts=experts, topk=rng.randint(1, min(16, experts)),
                    dtype=dtype, wdtype=rng.choice([dtype, "fp32"]), every=rng.random() < 0.5, wide=rng.random() < 0.5,
                    mask=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "layer":
        cols, hidden = _spread(rng, 64, 4096), _spread(rng, 32, 8192)
        gated = rng.random() < 0.7
        one = cols * hidden * (3 if gated else 2) * SIZE[dtype]
        experts = _spread(rng, 2, int(max(2, min(256, MOST_WEIGHTS / one))))
        topk = rng.randint(1, min(8, experts))
        tokens = _spread(rng, 1, 64)
        return dict(op=op, tokens=tokens, topk=topk, experts=experts, cols=cols, hidden=hidden, dtype=dtype,
                    wdtype=rng.choice([dtype, "fp32"]), gated=gated, act=rng.choice(["silu", "gelu", "relu"]),
                    drop=rng.choice([0.0, 0.0, 0.1, 0.5]) if tokens >= 8 else 0.0)
    rows, cols = _spread(rng, 8, 4096), _spread(rng, 8, 4096)
    case = dict(op=op, batch=1, rows=rows, cols=cols, dtype=dtype, gap=rng.choice([0, 0, 8, 13]))
    room = min(MOST_FLOPS / (2 * work(case)["flops"]), 1e8 / (rows * cols))
    case["batch"] = _spread(rng, 1, int(max(1, min(64, room))))
    return case


def _active(case):
    """The experts that get a token, on average over routings without a preference."""
    kept = case["tokens"] * (1 - case["drop"])
    return case["experts"] * (1 - (1 - case["topk"] / case["experts"]) ** kept)


def work(case):
    op, es = case["op"], SIZE[case["dtype"]]
    if op == "orthogonalize":
        # A and A^2 are symmetric: half of each product.
        m, n = sorted((case["rows"], case["cols"]))
        return {"bytes": 2 * case["batch"] * m * n * es, "flops": STEPS * case["batch"] * (3 * m * m * n + m ** 3)}
    tokens, topk, ws = case["tokens"], case["topk"], SIZE[case["wdtype"]]
    if op == "layer":
        one = case["cols"] * case["hidden"] * (3 if case["gated"] else 2)
        return {"bytes": _active(case) * one * es + 2 * tokens * case["cols"] * es + tokens * topk * (4 + ws),
                "flops": 2 * tokens * topk * (1 - case["drop"]) * one}
    row, ids = case["experts"] * es, tokens * topk * (8 if case["wide"] else 4)
    if op == "route":
        return {"bytes": tokens * row + ids + tokens * topk * ws, "flops": 4 * tokens * case["experts"]}
    read = tokens * row if case["every"] else tokens * topk * es
    return {"bytes": tokens * row + read + ids + tokens * topk * ws, "flops": 4 * tokens * case["experts"]}


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _logits(gen, case):
    """Scores of experts of different popularity; masked ones are -inf, and with a mask some tokens (padding of the batch)
    have nothing to choose."""
    tokens, experts = case["tokens"], case["experts"]
    x = 1.5 * _randn(gen, tokens, experts) + 0.5 * _randn(gen, experts)
    if case["mask"]:
        x[torch.rand(tokens, experts, generator=gen, device="cuda") < case["mask"]] = -math.inf
        x[torch.rand(tokens, generator=gen, device="cuda") < 0.05] = -math.inf
    return x.to(TYPES[case["dtype"]])


def _choose(x, topk, every):
    """Ids (the lowest first among equal logits; -1 where nothing is left to choose) and weights in the type of x."""
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    best, ids = best[:, :topk], ids[:, :topk]
    there = best > -math.inf
    top = torch.where(there[:, :1], best[:, :1], 0.0)
    e = torch.exp(best - top)
    total = (torch.exp(x - top) if every else e).sum(1, keepdim=True)
    return torch.where(there, ids, -1), torch.where(there, e / total, 0.0)


def _layer_weights(gen, case):
    """Both projections of all experts, of the size that keeps the values' scale."""
    def one(rows, cols, dtype):
        w = torch.empty(case["experts"], rows, cols, dtype=TYPES[dtype], device="cuda")
        return w.normal_(0.0, cols ** -0.5, generator=gen)
    return (one(case["hidden"] * (2 if case["gated"] else 1), case["cols"], case["dtype"]),
            one(case["cols"], case["hidden"], case["dtype"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "orthogonalize":
        # A gradient: a sum over few directions beside noise, small values.
        batch, rows, cols = case["batch"], case["rows"], case["cols"]
        rank = max(1, min(rows, cols) // 4)
        g = torch.randn(batch, rows, cols + case["gap"], generator=gen, device="cuda")
        g.baddbmm_(_randn(gen, batch, rows, rank), _randn(gen, batch, rank, cols + case["gap"]), beta=1.0, alpha=rank ** -0.5)
        s["g"] = g.mul_(1e-3).to(TYPES[case["dtype"]])[:, :, :cols]
        s["out"] = torch.zeros(batch, rows, cols, dtype=TYPES[case["dtype"]], device="cuda")
        return s
    tokens, topk, experts, wtype = case["tokens"], case["topk"], case["experts"], TYPES[case["wdtype"]]
    if op == "layer":
        s["x"] = _randn(gen, tokens, case["cols"]).to(TYPES[case["dtype"]])
        s["w_in"], s["w_out"] = _layer_weights(gen, case)
        ids, weights = _choose(_randn(gen, tokens, experts) + 0.2 * _randn(gen, experts), topk, False)
        if case["drop"]:
            ids[torch.rand(tokens, topk, generator=gen, device="cuda") < case["drop"]] = -1
        s["ids"], s["weights"] = ids.int(), weights.to(wtype)
        s["out"] = torch.zeros(tokens, case["cols"], dtype=TYPES[case["dtype"]], device="cuda")
        return s
    s["logits"] = x = _logits(gen, case)
    id_type = torch.int64 if case["wide"] else torch.int32
    if op == "route":
        s["ids"] = torch.zeros(tokens, topk, dtype=id_type, device="cuda")
        s["weights"] = torch.zeros(tokens, topk, dtype=wtype, device="cuda")
        return s
    s["ids"] = _choose(x.float(), topk, case["every"])[0].to(id_type)
    s["dweights"] = (0.1 * _randn(gen, tokens, topk)).to(wtype)
    s["dlogits"] = torch.zeros_like(x)
    return s


def _run_own(s):
    import allreduce_reduction_rank_gb300 as sar
    op = s["op"]
    if op == "orthogonalize":
        if "workspace" not in s:                        # kept by a program for all its calls
            n = sar.sar_orthogonalize_workspace_bytes(s["batch"], s["rows"], s["cols"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        sar.sar_orthogonalize(s["g"], s["out"], s["workspace"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return {"out": s["out"]}
    if op == "layer":
        if "workspace" not in s:
            n = sar.sar_expert_layer_workspace_bytes(s["tokens"], s["topk"], s["experts"], s["cols"], s["hidden"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        act = {"silu": sar.SAR_ACT_SILU, "gelu": sar.SAR_ACT_GELU, "relu": sar.SAR_ACT_RELU}[s["act"]]
        sar.sar_expert_layer(s["x"], s["ids"], s["w_in"], s["w_out"], s["out"], s["weights"], activation=act,
                             workspace=s["workspace"])
        return {"out": s["out"]}
    softmax = sar.SAR_SOFTMAX_ALL if s["every"] else sar.SAR_SOFTMAX_CHOSEN
    if op == "route":
        sar.sar_expert_route(s["logits"], s["ids"], s["weights"], softmax=softmax)
        return {"ids": s["ids"], "weights": s["weights"]}
    sar.sar_expert_route_backward(s["dweights"], s["logits"], s["ids"], s["dlogits"], softmax=softmax)
    return {"dlogits": s["dlogits"]}


def _activate(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return torch.where(z > 0, z, 0.0)


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "orthogonalize":
        a, b, c = COEFFICIENTS
        x = s["g"].float()
        x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + EPS)
        tall = s["rows"] > s["cols"]
        x = x.transpose(1, 2) if tall else x
        for _ in range(STEPS):
            gram = torch.bmm(x, x.transpose(1, 2))
            x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
        return {"out": (x.transpose(1, 2) if tall else x).to(s["g"].dtype).contiguous()}
    if op == "layer":
        hidden, experts, tokens, topk = s["hidden"], s["experts"], s["tokens"], s["topk"]
        if tokens * topk <= experts:
            # Few choices: each one's matrices, picked out.
            at = s["ids"].view(-1).clamp(min=0).long()
            rows = s["x"].float().repeat_interleave(topk, 0)[:, :, None]
            z = torch.bmm(s["w_in"][at].float(), rows)[:, :, 0]
            h = _activate(z[:, :hidden], s["act"])
            h = h * z[:, hidden:] if s["gated"] else h
            weight = torch.where(s["ids"] >= 0, s["weights"].float(), 0.0)
            y = torch.bmm(s["w_out"][at].float(), h[:, :, None]).view(tokens, topk, -1) * weight[:, :, None]
            return {"out": y.sum(1).to(s["x"].dtype)}
        # Every expert for every token; what a token did not choose has the weight 0.
        z = torch.matmul(s["x"].float(), s["w_in"].float().transpose(1, 2))                 # experts, tokens, hidden
        h = _activate(z[:, :, :hidden], s["act"])
        h = h * z[:, :, hidden:] if s["gated"] else h
        chosen = s["ids"][None] == torch.arange(experts, device="cuda", dtype=torch.int32)[:, None, None]
        weight = torch.where(chosen, s["weights"].float()[None], 0.0).sum(2)                # experts, tokens
        y = torch.bmm(h * weight[:, :, None], s["w_out"].float().transpose(1, 2))
        return {"out": y.sum(0).to(s["x"].dtype)}
    x = s["logits"].float()
    if op == "route":
        ids, weights = _choose(x, s["topk"], s["every"])
        return {"ids": ids.to(s["ids"].dtype), "weights": weights.to(s["weights"].dtype)}
    ids = s["ids"].long()
    there = (ids >= 0).float()
    top = x.max(1, keepdim=True).values
    top = torch.where(top > -math.inf, top, 0.0)
    picked = torch.exp(x.gather(1, ids.clamp(min=0)) - top) * there
    every = torch.exp(x - top)
    total = (every if s["every"] else picked).sum(1, keepdim=True)
    p = picked / torch.where(total > 0, total, 1.0)
    dw = s["dweights"].float()
    down = (p * dw).sum(1, keepdim=True)
    if s["every"]:
        out = -down * every / torch.where(total > 0, total, 1.0)
        out.scatter_add_(1, ids.clamp(min=0), p * dw)
    else:
        out = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), p * (dw - down) * there)
    return {"dlogits": out.to(s["logits"].dtype)}


def exact(case, seed):
    """The outputs from the definitions in 64 bits; ids are whole numbers and have none."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "orthogonalize":
        a, b, c = COEFFICIENTS
        x = s["g"].double()
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
        flip = case["rows"] > case["cols"]
        for _ in range(STEPS):                          # a x + A (b x + c A x), the Gram matrix on the short side
            t = x.mT
            if flip:
                gram = torch.matmul(t, x)
                x = a * x + torch.matmul(b * x + c * torch.matmul(x, gram), gram)
            else:
                gram = torch.matmul(x, t)
                x = a * x + torch.matmul(gram, b * x + c * torch.matmul(gram, x))
        return {"out": x}
    if op == "layer":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        for e in torch.unique(s["ids"]).tolist():       # one expert at a time, for the tokens that chose it
            if e < 0:
                continue
            t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
            z = s["x"][t].double() @ s["w_in"][e].double().T
            g = z[:, :case["hidden"]]
            if case["act"] == "silu":
                h = g * torch.special.expit(g)
            elif case["act"] == "gelu":
                h = g * torch.special.ndtr(g)
            else:
                h = g.clamp(min=0)
            if case["gated"]:
                h = h * z[:, case["hidden"]:]
            out.index_add_(0, t, (h @ s["w_out"][e].double().T) * s["weights"][t, j, None].double())
        return {"out": out}
    x = s["logits"].double()
    empty = (x == -math.inf).all(1, keepdim=True)
    x = torch.where(empty, 0.0, x)
    if op == "route":
        best = torch.topk(x, case["topk"], dim=1).values
        logs = best - torch.logsumexp(x if case["every"] else best, dim=1, keepdim=True)
        return {"ids": None, "weights": torch.where(empty, 0.0, torch.exp(logs))}
    ids, dw = s["ids"].long(), s["dweights"].double()
    there = ids >= 0
    chosen = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), there.double()) > 0
    given = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), torch.where(there, dw, 0.0))
    p = torch.softmax(x if case["every"] else torch.where(chosen, x, -math.inf), dim=1)
    p = torch.where(empty, 0.0, p)
    return {"dlogits": p * (given - (p * given).sum(1, keepdim=True))}
