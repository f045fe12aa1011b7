"""Plain 64-bit definitions of the operators around the allreduce, and the
error bounds that binary32 kernels of them keep to.

The bounds are first-order rounding analysis: U = 2^-24 is the unit roundoff of
binary32, OUT[dtype] that of the output's rounding, and a sum of n terms whose
longest chain of additions has `depth` of them is within depth * U of the sum of
the terms' magnitudes.  A row's sum runs over at least 32 threads, so its chain
is at most cols / 32 + 16 long; the sums over rows are split into at least
min(rows, 64) shares of equal size and those added: rows / 64 + 400.  SLACK
covers the second-order terms.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
OUT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
SLACK = 1.25
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def row_depth(cols):
    return cols / 32 + 16


def column_depth(rows):
    return rows / 64 + 400


def check(got, want, bound, what=""):
    """|got - want| within the bound, element by element; NaN and infinities where want has them."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: other elements are finite"
    assert torch.equal(torch.isnan(want), torch.isnan(got)), f"{what}: other elements are NaN"
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]), f"{what}: infinities differ"
    off = ((got - want).abs() - bound)[fine]
    worst = off.max().item() if off.numel() else -1.0
    assert worst <= 0, f"{what}: over its bound by {worst:.3g}"


def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) in 64 bits and the bounds of the three (y's without the output's rounding)."""
    x = x.double()
    n = x.shape[1]
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(n, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    h = d * rstd
    y = h * w + b
    gamma = (row_depth(n) + 2) * U
    e_mean = gamma * x.abs().mean(1, keepdim=True)
    rel = 0.5 * (gamma + 6 * U + e_mean ** 2 / (var + eps).clamp(min=1e-300)) + 4 * U
    e_h = rstd * (e_mean + U * d.abs()) + h.abs() * (rel + U)
    e_y = w.abs() * e_h + U * y.abs()
    return (y, mean.view(-1), rstd.view(-1)), (SLACK * e_y, SLACK * e_mean.view(-1), SLACK * (rel * rstd).view(-1))


def layer_norm_backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) in 64 bits and their bounds, without the outputs' rounding."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, n = x.shape
    w = torch.ones(n, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    h, g = (x - mean) * rstd, dy * w
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - mg - h * mgh)
    gamma = (row_depth(n) + 6) * U
    e_mg, e_mgh = gamma * g.abs().mean(1, keepdim=True), gamma * (g * h).abs().mean(1, keepdim=True)
    e_dx = rstd * (e_mg + h.abs() * e_mgh + 6 * U * (g.abs() + mg.abs() + (h * mgh).abs())) + U * dx.abs()
    down = (column_depth(rows) + 4) * U
    return ((dx, (dy * h).sum(0), dy.sum(0)),
            (SLACK * e_dx, SLACK * down * (dy * h).abs().sum(0), SLACK * down * dy.abs().sum(0)))


def rounded(bound, want, dtype):
    """The bound with the rounding of the output to dtype."""
    return bound + OUT[dtype] * (want.abs() + bound) + TINY[dtype]


def expert_sort(ids, experts, align, capacity):
    """counts, offsets, position, source of a list of lists of ids, one slot at a time."""
    counts = [0] * experts
    for row in ids:
        for e in row:
            if 0 <= e < experts:
                counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    nxt, position, source = offsets[:-1].copy(), [], [-1] * capacity
    topk = len(ids[0]) if ids else 1
    for t, row in enumerate(ids):
        position.append([])
        for j, e in enumerate(row):
            p = -1
            if 0 <= e < experts:
                p = nxt[e]
                nxt[e] += 1
                if p >= capacity:
                    p = -1
                else:
                    source[p] = t * topk + j
            position[-1].append(p)
    return counts, offsets, position, source


def combine(rows, position, weights):
    """out in 64 bits and its bound."""
    kept = position >= 0
    picked = torch.where(kept[:, :, None], rows[position.clamp(min=0).long()].double(), 0.0)
    if weights is not None:
        picked = picked * torch.where(kept, weights.double(), 0.0)[:, :, None]
    return picked.sum(1), SLACK * (position.shape[1] + 1) * U * picked.abs().sum(1)


def combine_backward(dout, rows, position, weights, capacity):
    """(drows with zeros where no slot is, dweights) in 64 bits and their bounds."""
    tokens, topk = position.shape
    kept = position >= 0
    d = dout.double()
    picked = torch.where(kept[:, :, None], rows[position.clamp(min=0).long()].double(), 0.0)
    terms = torch.where(kept[:, :, None], picked * d[:, None, :], 0.0)
    drows = torch.zeros(capacity, dout.shape[1], dtype=torch.float64, device=dout.device)
    t, j = torch.nonzero(kept, as_tuple=True)
    drows[position[t, j].long()] = d[t] * weights.double()[t, j][:, None]
    return ((drows, terms.sum(2)),
            (SLACK * U * drows.abs(), SLACK * (row_depth(dout.shape[1]) + 2) * U * terms.abs().sum(2)))
