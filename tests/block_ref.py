"""Plain 64-bit definitions of the router, the expert layer of a few tokens and
the Newton-Schulz iteration, and the error bounds that binary32 kernels of them
keep to (first-order rounding analysis, as in tests/operator_ref.py: U = 2^-24,
SLACK for the second-order terms).

CUDA documents expf, erff and erfcf to 2, 2 and 4 units in the last place of
binary32; a unit in the last place is at most 2 U of the value.
"""
from __future__ import annotations

import math

import torch

from tests.operator_ref import SLACK, U


def route(logits, topk, every):
    """ids (lists), weights in 64 bits and their bounds, one token at a time on the CPU."""
    x = logits.detach().cpu().double()
    ids, weights, bounds = [], [], []
    for row in x.tolist():
        order = sorted(range(len(row)), key=lambda e: (-(math.inf if math.isnan(row[e]) else row[e]), not math.isnan(row[e]), e))
        chosen = [e for e in order[:topk] if row[e] != -math.inf]
        counted = [row[e] for e in (range(len(row)) if every else chosen) if row[e] != -math.inf]
        w, b = [], []
        bad = any(math.isnan(v) or v == math.inf for v in counted)
        top = max(counted) if counted and not bad else 0.0
        total = sum(math.exp(v - top) for v in counted) if not bad else math.nan
        # the argument's rounding |v - top| U, expf 4 U, and len / 32 + 6 additions of a sum over the lanes
        rel = (sum(math.exp(v - top) * (abs(v - top) + 4) for v in counted) / total if counted and not bad else 0.0) + \
            len(counted) / 32 + 6
        for e in chosen:
            p = math.exp(row[e] - top) / total if not bad else math.nan
            w.append(p)
            b.append(0.0 if bad else SLACK * U * p * (rel + abs(row[e] - top) + 4 + 1))
        pad = topk - len(chosen)
        ids.append(chosen + [-1] * pad)
        weights.append(w + [0.0] * pad)
        bounds.append(b + [0.0] * pad)
    return ids, torch.tensor(weights, dtype=torch.float64), torch.tensor(bounds, dtype=torch.float64)


def route_backward(dweights, logits, ids, every):
    """dlogits in 64 bits and its bound; ids outside the experts are dropped, equal ones add up."""
    x, dw = logits.double(), dweights.double()
    tokens, experts = x.shape
    there = (ids >= 0) & (ids < experts)
    at = torch.where(there, ids.long(), 0)
    g = torch.zeros_like(x).scatter_add_(1, at, torch.where(there, dw, 0.0))
    ga = torch.zeros_like(x).scatter_add_(1, at, torch.where(there, dw.abs(), 0.0))
    chosen = torch.zeros_like(x).scatter_add_(1, at, there.double()) > 0
    counted = torch.where(chosen | torch.tensor(every, device=x.device), x, -math.inf)
    top = counted.max(1, keepdim=True).values
    empty = top == -math.inf
    d = counted - torch.where(empty, 0.0, top)
    e = torch.where(empty | (counted == -math.inf), 0.0, torch.exp(d))
    total = torch.where(empty, 1.0, e.sum(1, keepdim=True))
    p = e / total
    s = (p * g).sum(1, keepdim=True)
    out = p * torch.where(torch.isnan(p) & ~chosen, -s, g - s)
    if not every:
        out = torch.where(chosen, out, 0.0)
    arg = torch.where(torch.isfinite(d), d.abs(), 0.0) + 4          # relative error of exp, in U
    rel = arg + (p * arg).sum(1, keepdim=True) + experts / 32 + 10
    e_s = (p * ga * (rel + 8)).sum(1, keepdim=True) * U
    bound = p * ((rel + 2) * U * (g.abs() + s.abs()) + 32 * U * ga + e_s)
    return out, SLACK * torch.nan_to_num(bound)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    return torch.where(z <= 0, 0.0, z)


def expert_layer(x, ids, w_in, w_out, weights, gated, act):
    """out in 64 bits and its bound without the output's rounding.

    A product's sum may run in steps of 16 terms whose binary32 accumulator is off by up to two units in the last place
    (4 U) each, so K / 4 U of the terms' magnitudes, and 32 U more for the joins; two factors held as two numbers of 10 or
    more bits each leave 12 U.  The activations' slope is at most 1.13, their own error 16 U.  h as two numbers of 8 bits
    (bf16) is off by 2^-16 at most.
    """
    tokens, topk = ids.shape
    experts, hidden = w_in.shape[0], w_out.shape[2]
    cols = x.shape[1]
    out = torch.zeros(tokens, cols, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    d_in, d_out = (cols / 4 + 44) * U, (hidden / 4 + 44) * U
    split = 2.0 ** -16 if x.dtype == torch.bfloat16 else 2.0 ** -21
    for t in range(tokens):
        for j in range(topk):
            e = int(ids[t, j])
            if not 0 <= e < experts:
                continue
            xi, wi, wo = x[t].double(), w_in[e].double(), w_out[e].double()
            z, ez = wi @ xi, d_in * (wi.abs() @ xi.abs())
            g = _act(z[:hidden], act)
            eg = 1.13 * ez[:hidden] + 16 * U * g.abs()
            if gated:
                h, eh = g * z[hidden:], eg * z[hidden:].abs() + (g.abs() + eg) * ez[hidden:]
            else:
                h, eh = g, eg
            eh = eh + (2 * U + split) * h.abs()
            y = wo @ h
            ey = wo.abs() @ eh + d_out * (wo.abs() @ h.abs())
            w = 1.0 if weights is None else float(weights[t, j])
            out[t] += w * y
            bound[t] += abs(w) * (ey + (topk + 2) * U * y.abs())
    return out, SLACK * bound


def newton_schulz(g, steps, coefficients, eps, scale=1.0, noise=0.0, seed=0):
    """The iteration of a batch in 64 bits.  With `noise`, every product's elements are off by up to noise * U of the sum of
    their terms' magnitudes, at random, and so is the beginning: what a computation in binary32 does."""
    a, b, c = coefficients
    gen = torch.Generator(device=g.device).manual_seed(seed)

    def off(value, magnitude):
        if not noise:
            return value
        return value + noise * U * magnitude * (2 * torch.rand(value.shape, generator=gen, device=g.device, dtype=torch.float64) - 1)

    def product(p, q):
        return off(p @ q, p.abs() @ q.abs())
    x = g.double()
    tall = x.shape[1] > x.shape[2]
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + eps)
    x = x.mT if tall else x
    x = off(x, x.abs())
    for _ in range(steps):
        gram = product(x, x.mT)
        square = product(gram, gram)
        poly = off(b * gram + c * square, (b * gram).abs() + (c * square).abs())
        mix = product(poly, x)
        x = off(a * x + mix, (a * x).abs() + mix.abs())
    return scale * (x.mT if tall else x)


def newton_schulz_bound(g, steps, coefficients, eps, scale=1.0):
    """How far a result may be from newton_schulz's, matrix by matrix, as 2-norm of the difference over that of the values.

    The steps multiply errors by up to a each, so a bound by worst cases says nothing; the errors of a binary32 computation
    are put into the 64-bit one instead.  An element's error is at most 4 U of its terms' magnitudes for operands held as
    two numbers of 11 bits (3 U) and short chains of additions joined in binary32; its size is drawn up to 8 U, and the
    bound is three times the worst of three such runs."""
    want = newton_schulz(g, steps, coefficients, eps, scale)
    worst = torch.zeros(g.shape[0], dtype=torch.float64, device=g.device)
    for seed in range(3):
        other = newton_schulz(g, steps, coefficients, eps, scale, noise=8.0, seed=seed)
        worst = torch.maximum(worst, (other - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1).clamp(min=1e-300))
    return want, 3 * worst
