"""One data-parallel training step of a block with experts over simulated ranks.

    python -m allreduce_reduction_rank_gb300.block_step [--ranks 4] [--tokens 512] [--cols 1024] [--experts 16]
                                                         [--topk 2] [--dtype bf16]

Each rank has its own tokens; all have the same parameters.  A rank's step is

    h = layer norm(x);  ids, weights = the router's best choices for h
    sort the choices by expert;  rows = h dispatched;  rows' = rows @ the expert's matrix, segment by segment
    y = x + combine(rows', weights)

and back again for a given gradient of y.  The gradients of the parameters (layer norm's weight and bias, the router,
the experts) are then summed over the ranks by one allreduce, and every rank takes the same update from them: matrices
(each expert's, the router's) in the orthogonalised direction of their gradient, vectors along it.  Layer norm, the
router's choice (of up to 32 experts a token; torch's beyond), sort, dispatch, combine, their gradients, the allreduce and
the orthogonalisation are this library's calls; the matrix products are torch's.  The command checks every rank's sums against torch.autograd on the same step in
64 bits, and the update against the same iteration in 64 bits, and prints how far they are off.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

import allreduce_reduction_rank_gb300 as sar

#: Rows that an expert's segment is padded to a multiple of: a matrix product's tile.
ALIGN = 16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@dataclass
class Parameters:
    norm_weight: torch.Tensor      # (cols), float32
    norm_bias: torch.Tensor        # (cols), float32
    router: torch.Tensor           # (cols, experts), float32
    experts: torch.Tensor          # (experts, cols, cols), the rows' type

    @staticmethod
    def random(cols: int, experts: int, dtype: torch.dtype, seed: int = 0) -> "Parameters":
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")
        return Parameters(1 + 0.1 * randn(cols), 0.1 * randn(cols), randn(cols, experts) / cols ** 0.5,
                          (randn(experts, cols, cols) / cols ** 0.5).to(dtype))


class RankStep:
    """One rank's buffers, kept from step to step, and its step."""

    def __init__(self, tokens: int, params: Parameters, topk: int):
        cols, experts = params.router.shape
        dtype = params.experts.dtype
        self.params, self.topk = params, topk
        self.capacity = sar.sar_expert_rows(tokens, topk, experts, ALIGN)
        new = dict(device="cuda")
        self.h = torch.empty(tokens, cols, dtype=dtype, **new)
        self.mean, self.rstd = torch.empty(tokens, **new), torch.empty(tokens, **new)
        self.counts = torch.empty(experts, dtype=torch.int32, **new)
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, **new)
        self.position = torch.empty(tokens, topk, dtype=torch.int32, **new)
        self.dscores = torch.empty(tokens, experts, **new)
        # Segments of this step: rows past the last one are never read.
        self.rows, self.made = (torch.empty(self.capacity, cols, dtype=dtype, **new) for _ in range(2))
        self.dmade, self.drows = (torch.empty(self.capacity, cols, dtype=dtype, **new) for _ in range(2))
        self.out, self.dh, self.dx = (torch.empty(tokens, cols, dtype=dtype, **new) for _ in range(3))
        self.dweights = torch.empty(tokens, topk, **new)
        self.workspace = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(tokens, cols), dtype=torch.uint8, **new)
        # All gradients of the parameters in one buffer, for one allreduce.
        sizes = [cols, cols, cols * experts, experts * cols * cols]
        self.gradients = torch.zeros(sum(sizes), **new)
        self.dnorm_weight, self.dnorm_bias, drouter, dexperts = torch.split(self.gradients, sizes)
        self.drouter, self.dexperts = drouter.view(cols, experts), dexperts.view(experts, cols, cols)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        p = self.params
        sar.sar_layer_norm(x, self.h, p.norm_weight, p.norm_bias, self.mean, self.rstd)
        self.scores = self.h.float() @ p.router
        self.choose()
        sar.sar_expert_sort(self.ids, self.counts, self.offsets, self.position, align=ALIGN, capacity=self.capacity)
        sar.sar_expert_dispatch(self.h, self.position, self.rows, self.counts, self.offsets)
        self.segments = list(zip(self.offsets.tolist(), self.offsets.tolist()[1:]))
        for e, (a, b) in enumerate(self.segments):
            torch.matmul(self.rows[a:b], p.experts[e], out=self.made[a:b])
        sar.sar_expert_combine(self.made, self.position, self.out, self.weights)
        return x + self.out

    def choose(self) -> None:
        """The tokens' ids and weights from their scores; new tensors, which the next step leaves alone."""
        if self.topk > sar.SAR_MAX_TOPK:                     # more than the router makes
            best, self.ids = torch.topk(self.scores, self.topk, dim=1)
            self.weights = torch.softmax(best, dim=1)
            return
        shape = self.scores.shape[0], self.topk
        self.ids, self.weights = torch.empty(shape, dtype=torch.int64, device="cuda"), torch.empty(shape, device="cuda")
        sar.sar_expert_route(self.scores, self.ids, self.weights)

    def choose_backward(self) -> None:
        """The scores' gradient from the weights'."""
        if self.topk > sar.SAR_MAX_TOPK:
            dbest = self.weights * (self.dweights - (self.weights * self.dweights).sum(1, keepdim=True))
            self.dscores.zero_().scatter_(1, self.ids, dbest)
            return
        sar.sar_expert_route_backward(self.dweights, self.scores, self.ids, self.dscores)

    def backward(self, x: torch.Tensor, dy: torch.Tensor) -> torch.Tensor:
        p = self.params
        sar.sar_expert_combine_backward(dy, self.made, self.position, self.weights, self.dmade, self.dweights, self.counts,
                                        self.offsets)
        for e, (a, b) in enumerate(self.segments):
            torch.matmul(self.dmade[a:b], p.experts[e].T, out=self.drows[a:b])
            self.dexperts[e] = self.rows[a:b].float().T @ self.dmade[a:b].float()
        sar.sar_expert_combine(self.drows, self.position, self.dh)                # the dispatch's gradient
        # through the softmax of the chosen scores to the router
        self.choose_backward()
        self.drouter.copy_(self.h.float().T @ self.dscores)
        dh = (self.dh.float() + self.dscores @ p.router.T).to(x.dtype)
        sar.sar_layer_norm_backward(dh, x, p.norm_weight, self.mean, self.rstd, self.dx, self.dnorm_weight, self.dnorm_bias,
                                    workspace=self.workspace)
        return self.dx + dy


def step(ranks, xs, dys):
    """Every rank's forward and backward pass, then the allreduce of the gradients: (ys, dxs, sums), a sum for each rank."""
    ys = [r.forward(x) for r, x in zip(ranks, xs)]
    dxs = [r.backward(x, dy) for r, x, dy in zip(ranks, xs, dys)]
    sums = [torch.empty_like(r.gradients) for r in ranks]
    sar.sar_allreduce([r.gradients for r in ranks], sums)
    return ys, dxs, sums


class Update:
    """The parameters' update from a sum of gradients (a RankStep's layout), with its buffers kept."""

    def __init__(self, params: Parameters, rate: float = 0.02):
        self.rate = rate
        cols, experts = params.router.shape
        self.shapes = [(cols,), (cols,), (cols, experts), (experts, cols, cols)]
        self.router, self.experts = (torch.empty(s, device="cuda") for s in self.shapes[2:])
        n = max(sar.sar_orthogonalize_workspace_bytes(1, cols, experts), sar.sar_orthogonalize_workspace_bytes(experts, cols, cols))
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")

    def directions(self, total: torch.Tensor):
        """What each parameter moves against: vectors' gradients as they are, matrices' orthogonalised, with the scale that
        gives a tall matrix's rows the length of a square one's."""
        parts = torch.split(total, [torch.Size(s).numel() for s in self.shapes])
        dweight, dbias, drouter, dexperts = (p.view(s) for p, s in zip(parts, self.shapes))
        rows, cols = self.shapes[2]
        sar.sar_orthogonalize(drouter, self.router, self.workspace, scale=max(1.0, rows / cols) ** 0.5)
        sar.sar_orthogonalize(dexperts, self.experts, self.workspace)
        return dweight, dbias, self.router, self.experts

    def apply(self, params: Parameters, total: torch.Tensor) -> None:
        """Moves the parameters, in place."""
        moved = (params.norm_weight, params.norm_bias, params.router, params.experts)
        for p, d in zip(moved, self.directions(total)):
            p.sub_((self.rate * d).to(p.dtype))


def orthogonal_reference(g, scale=1.0):
    """sar_orthogonalize's iteration in 64 bits."""
    x = g.double()
    x = x / (x.flatten(-2).norm(dim=-1)[..., None, None] + 1e-7)
    x = x.mT if g.shape[-2] > g.shape[-1] else x
    for _ in range(5):
        gram = x @ x.mT
        x = 3.4445 * x + (-4.7750 * gram + 2.0315 * gram @ gram) @ x
    return scale * (x.mT if g.shape[-2] > g.shape[-1] else x)


def reference(params: Parameters, x, dy, ids):
    """One rank's y, dx and gradients by torch.autograd in 64 bits, for the same choices of experts."""
    leaves = [t.double().requires_grad_() for t in (params.norm_weight, params.norm_bias, params.router, params.experts)]
    nw, nb, router, experts = leaves
    xd = x.double().requires_grad_()
    h = (xd - xd.mean(1, keepdim=True)) * (xd.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * nw + nb
    weights = torch.softmax((h @ router).gather(1, ids), dim=1)
    y = xd
    for j in range(ids.shape[1]):
        made = torch.zeros_like(h)
        for e in range(experts.shape[0]):
            mine = torch.nonzero(ids[:, j] == e).view(-1)
            made = made.index_add(0, mine, h[mine] @ experts[e])
        y = y + weights[:, j, None] * made
    grads = torch.autograd.grad(y, [xd] + leaves, dy.double())
    return y.detach(), grads[0], torch.cat([g.reshape(-1) for g in grads[1:]])


def deviation(got: torch.Tensor, want: torch.Tensor) -> float:
    """2-norm of the difference over that of the values."""
    return ((got.double() - want).norm() / want.norm()).item()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--cols", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--topk", type=int, default=2)
    ap.add_argument("--dtype", choices=sorted(TYPES), default="bf16")
    a = ap.parse_args()
    torch.cuda.set_device(0)
    dtype = TYPES[a.dtype]
    params = Parameters.random(a.cols, a.experts, dtype)
    ranks = [RankStep(a.tokens, params, a.topk) for _ in range(a.ranks)]
    g = torch.Generator(device="cuda").manual_seed(1)
    xs, dys = ([torch.randn(a.tokens, a.cols, generator=g, device="cuda").to(dtype) for _ in ranks] for _ in range(2))
    ys, dxs, sums = step(ranks, xs, dys)
    want = [reference(params, x, dy, r.ids) for x, dy, r in zip(xs, dys, ranks)]
    total = sum(w[2] for w in want)
    print(f"block_step: {a.ranks} ranks, {a.tokens} tokens x {a.cols}, {a.topk} of {a.experts} experts, {a.dtype}")
    print("  relative deviation from 64 bits: y %.2g, dx %.2g, summed gradients %.2g" % (
        max(deviation(y, w[0]) for y, w in zip(ys, want)), max(deviation(d, w[1]) for d, w in zip(dxs, want)),
        max(deviation(s, total) for s in sums)))
    if not all(torch.equal(s, sums[0]) for s in sums):
        raise SystemExit("block_step: the ranks' sums differ")
    update = Update(params)
    _, _, router, expert_matrices = update.directions(sums[0])
    drouter, dexperts = (p.view(s) for p, s in zip(torch.split(sums[0][2 * a.cols:], [router.numel(), expert_matrices.numel()]),
                                                   update.shapes[2:]))
    scale = max(1.0, a.cols / a.experts) ** 0.5
    print("  update: router %.2g, experts %.2g" % (deviation(router, orthogonal_reference(drouter, scale)),
                                                 deviation(expert_matrices, orthogonal_reference(dexperts))))
    update.apply(params, sums[0])


if __name__ == "__main__":
    main()
