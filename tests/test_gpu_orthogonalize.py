"""The Newton-Schulz iteration (sar_orthogonalize) against the same in 64 bits,
within what binary32's roundings do to it (tests/block_ref.py)."""
import math

import pytest
import torch

from tests import block_ref as bref
from tests import operator_ref as ref

pytestmark = pytest.mark.gpu
MARK = 3.0
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def gradients(batch, rows, cols, dtype, seed=0, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rank = max(1, min(rows, cols) // 4)
    x = torch.randn(batch, rows, cols, generator=g, device="cuda")
    x += torch.randn(batch, rows, rank, generator=g, device="cuda") @ torch.randn(batch, rank, cols, generator=g, device="cuda")
    return (scale * x).to(dtype)


def laid(values, gap=0, between=0, offset=0):
    """A copy of a batch with leading dimension cols + gap and `between` more elements between the matrices."""
    batch, rows, cols = values.shape
    ld = cols + gap
    stride = rows * ld + between
    flat = torch.full((offset + batch * stride + 64,), MARK, dtype=values.dtype, device="cuda")
    view = flat[offset:].as_strided((batch, rows, cols), (stride, ld, 1), offset)
    view.copy_(values)
    return view, flat


def run(sar, g, steps=5, coefficients=MUON, eps=1e-7, scale=1.0, inplace=False, **layout):
    gv, _ = laid(g, **layout)
    ov, flat = (gv, None) if inplace else laid(torch.zeros_like(g), **layout)
    need = sar.sar_orthogonalize_workspace_bytes(*g.shape)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")            # NaN all over
    sar.sar_orthogonalize(gv, ov, ws[:need], steps=steps, coefficients=coefficients, eps=eps, scale=scale)
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    got = ov.clone()
    if flat is not None:
        ov.fill_(MARK)
        assert bool((flat == MARK).all())
    return got


def check(sar, g, steps=5, coefficients=MUON, eps=1e-7, scale=1.0, **layout):
    got = run(sar, g, steps, coefficients, eps, scale, **layout).double()
    want, bound = bref.newton_schulz_bound(g, steps, coefficients, eps, scale)
    off = (got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    # beside the rounding of the output, at most OUT of each element (TINY where that is subnormal)
    allowed = bound + ref.OUT[g.dtype] + ref.TINY[g.dtype] * math.sqrt(want[0].numel()) / want.flatten(1).norm(dim=1)
    assert bool((off <= allowed).all()), (off.max().item(), allowed.min().item())


SIZES = [(1, 1, 1), (1, 1, 7), (3, 5, 1), (2, 8, 8), (1, 16, 33), (5, 31, 17), (2, 64, 64), (1, 100, 60), (8, 128, 128),
         (2, 128, 200), (1, 129, 128), (1, 130, 300), (2, 256, 64), (1, 257, 255), (1, 500, 130), (1, 64, 1000), (1, 1003, 97),
         (1, 384, 640), (40, 24, 56), (1, 512, 512), (1, 8, 3648), (2, 4096, 100), (1, 4097, 100), (3, 65, 513), (1, 128, 1030),
         (200, 16, 16)]


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("batch,rows,cols", SIZES)
def test_orthogonalize(sar, batch, rows, cols, dtype):
    check(sar, gradients(batch, rows, cols, ref.DTYPES[dtype], seed=rows + cols))


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("batch,rows,cols", [(70, 256, 250), (12, 600, 600), (6, 600, 1000), (6, 1000, 600), (100, 130, 128),
                                             (40, 200, 400), (1, 2600, 2700)])
def test_many_tiles(sar, batch, rows, cols, dtype):
    """Enough of them that pairs of blocks take some of the products, or all."""
    check(sar, gradients(batch, rows, cols, ref.DTYPES[dtype], seed=rows), steps=2 if rows > 2000 else 5)


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("batch,rows,cols", [(9, 300, 640), (13, 300, 300), (14, 200, 257), (12, 300, 300), (1, 700, 660)])
def test_tiles_of_either_width(sar, batch, rows, cols, dtype):
    """About where the products' tiles of 64 columns outnumber the SMs: 9 x 3 x 10, 13 x 12, 14 x 2 x 5; and below."""
    check(sar, gradients(batch, rows, cols, ref.DTYPES[dtype], rows + batch))


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("batch,rows,cols", [(3, 20, 37), (2, 150, 77), (2, 130, 140)])
def test_layouts(sar, batch, rows, cols, dtype):
    g = gradients(batch, rows, cols, ref.DTYPES[dtype], seed=2)
    plain = run(sar, g)
    check(sar, g, gap=3, between=5, offset=1, scale=0.2)
    assert torch.equal(run(sar, g, gap=8, between=16), plain)
    assert torch.equal(run(sar, g, gap=1, offset=3), plain)
    assert torch.equal(run(sar, g, inplace=True, gap=5), plain)
    shared = g[:1].expand(batch, rows, cols)                                  # one matrix, read by all
    out = torch.empty_like(g)
    ws = torch.empty(sar.sar_orthogonalize_workspace_bytes(batch, rows, cols), dtype=torch.uint8, device="cuda")
    sar.sar_orthogonalize(shared, out, ws)
    assert all(torch.equal(out[i], plain[0]) for i in range(batch))
    two = torch.empty_like(g[0])
    sar.sar_orthogonalize(g[1], two, ws)                                      # a matrix without a batch
    assert torch.equal(two, plain[1])


@pytest.mark.parametrize("steps,coefficients", [(1, MUON), (2, MUON), (9, MUON), (12, (1.5, -0.5, 0.0)), (6, (1.875, -1.25, 0.375)),
                                                (3, (1.0, 0.0, 0.0)), (4, (1.0, 0.5, -0.5)), (3, (-2.0, 0.5, 0.25))])
@pytest.mark.parametrize("batch,rows,cols", [(2, 48, 80), (1, 200, 150)])
def test_steps_and_coefficients(sar, batch, rows, cols, steps, coefficients):
    check(sar, gradients(batch, rows, cols, torch.float32, seed=4), steps, coefficients)


def test_it_makes_matrices_orthogonal(sar):
    """With (1.875, -1.25, 0.375) the singular values go to 1: after 25 steps from a well-conditioned matrix X X^T = I."""
    g = torch.linalg.qr(torch.randn(2, 96, 96, generator=torch.Generator().manual_seed(1), dtype=torch.float64))[0].float().cuda()
    g = g + 0.1 * gradients(2, 96, 96, torch.float32, seed=5, scale=0.1)
    out = run(sar, g, steps=25, coefficients=(1.875, -1.25, 0.375)).double()
    assert (out @ out.mT - torch.eye(96, device="cuda")).abs().max() < 1e-5


@pytest.mark.parametrize("scale", [1e-36, 1e-20, 1e20, 1e37])
@pytest.mark.parametrize("rows,cols", [(40, 64), (140, 150)])
def test_gradients_of_any_magnitude(sar, rows, cols, scale):
    """The squares leave binary32's range, the result does not."""
    g = gradients(2, rows, cols, torch.float32, seed=6, scale=scale)
    check(sar, g, eps=0.0)
    check(sar, g)
    mixed = gradients(2, rows, cols, torch.float32, seed=7, scale=1.0)
    mixed[:, 0] *= 1e25
    check(sar, mixed, eps=0.0)


@pytest.mark.parametrize("dtype", list(ref.DTYPES))
@pytest.mark.parametrize("rows,cols", [(40, 64), (140, 150)])
def test_zeros_infinities_and_nan(sar, rows, cols, dtype):
    g = gradients(5, rows, cols, ref.DTYPES[dtype], seed=8)
    clean = run(sar, g)
    g[0] = 0
    g[1, 3, 2] = math.nan
    g[2, 0, 1] = -math.inf
    got = run(sar, g)
    assert not got[0].any() and torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    assert torch.equal(got[3:], clean[3:])
    assert torch.isnan(run(sar, g[:1], eps=0.0)).all()                        # 0 / 0


def test_empty(sar):
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        t = torch.zeros(shape, device="cuda")
        sar.sar_orthogonalize(t, t, ws)


def test_captured_twice_over_one_workspace(sar):
    gs = [gradients(2, 70, 130, torch.float32, 9), gradients(1, 300, 200, torch.bfloat16, 10), gradients(4, 32, 32, torch.float16, 11)]
    ws = torch.empty(max(sar.sar_orthogonalize_workspace_bytes(*g.shape) for g in gs), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(g) for g in gs], []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for g, out in zip(gs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            sar.sar_orthogonalize(g, out, ws)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for g, out in zip(gs, outs):
        assert torch.equal(out, run(sar, g))


def test_calls_at_once(sar):
    """On streams of their own, with workspaces of their own: one launch, clusters that share k, pairs and single blocks."""
    gs = [gradients(8, 128, 128, torch.float32, 12), gradients(1, 300, 1100, torch.float16, 13), gradients(1, 128, 4000, torch.bfloat16, 14),
          gradients(2, 1003, 357, torch.float16, 15), gradients(1, 1024, 1536, torch.bfloat16, 16), gradients(6, 16, 24, torch.float32, 17)]
    want = [run(sar, g) for g in gs]
    outs = [torch.empty_like(g) for g in gs]
    spaces = [torch.empty(sar.sar_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device="cuda") for g in gs]
    streams = [torch.cuda.Stream() for _ in gs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, out, ws, s in zip(gs, outs, spaces, streams):
            sar.sar_orthogonalize(g, out, ws, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_refusals(sar):
    g = gradients(2, 8, 12, torch.float32)
    out, ws = torch.empty_like(g), torch.empty(sar.sar_orthogonalize_workspace_bytes(2, 8, 12), dtype=torch.uint8, device="cuda")

    def call(g=g, out=out, ws=ws, **kw):
        sar.sar_orthogonalize(g, out, ws, **kw)
    call()
    for kw in (dict(out=out.half()), dict(out=out[:1]), dict(g=g.transpose(1, 2)), dict(g=g[0, 0]), dict(g=g.cpu()),
               dict(coefficients=(1.0, 2.0)), dict(ws=ws[::2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=math.nan), dict(scale=math.inf), dict(ws=ws[:-1]),
               dict(ws=ws[1:]), dict(ws=None), dict(coefficients=(5.0, 0.0, 0.0)), dict(coefficients=(math.nan, 0, 0)),
               dict(coefficients=(2.0, 0.0, 0.0)), dict(coefficients=(0.0, 0.0, 3.5)), dict(coefficients=(0.0, 1.0, 0.0)),
               dict(coefficients=(-0.99, 0.0, 0.0)), dict(coefficients=(1.0, math.inf, 0)), dict(out=out[:1].expand(2, 8, 12))):
        with pytest.raises((sar.SarError, ValueError) if kw.get("ws", ws) is None else sar.SarError):
            call(**kw)
