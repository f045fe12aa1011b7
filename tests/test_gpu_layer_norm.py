"""Layer norm and its gradient against 64-bit definitions, at the sizes,
layouts and values where the kernels change their way or can go wrong, with the
bounds of tests/operator_ref.py."""
import pytest
import torch

from tests import operator_ref as ref

pytestmark = pytest.mark.gpu
MARK = 3.0


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


def placed(values, gap=0, offset=0):
    """A copy of a matrix with leading dimension cols + gap that starts `offset`
    elements into a marked buffer; returns the view and the buffer."""
    rows, cols = values.shape
    ld = cols + gap
    flat = torch.full((offset + rows * ld + 64,), MARK, dtype=values.dtype, device="cuda")
    view = flat[offset: offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(values)
    return view, flat


def untouched(view, flat):
    """Every element of the buffer outside the view still holds the mark."""
    was = view.clone()
    view.fill_(MARK)
    ok = bool((flat == MARK).all())
    view.copy_(was)
    return ok


def inputs(rows, cols, dtype, wdtype, seed=0, spread=1.5, shift=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g, device="cuda") * spread + shift).to(dtype)
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(dtype)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(wdtype)
    b = (0.2 * torch.randn(cols, generator=g, device="cuda")).to(wdtype)
    return x, dy, w, b


def forward(sar, x, w, b, eps=1e-5, gap=0, offset=0):
    rows = x.shape[0]
    xv, xf = placed(x, gap, offset)
    yv, yf = placed(torch.zeros_like(x), gap, offset)
    mean, rstd = torch.full((rows,), MARK, device="cuda"), torch.full((rows,), MARK, device="cuda")
    sar.sar_layer_norm(xv, yv, w, b, mean, rstd, eps=eps)
    torch.cuda.synchronize()
    assert untouched(yv, yf) and torch.equal(xv.contiguous().view(torch.uint8), x.view(torch.uint8))
    return yv, mean, rstd


def check_forward(sar, x, w, b, eps=1e-5, gap=0, offset=0):
    y, mean, rstd = forward(sar, x, w, b, eps, gap, offset)
    (wy, wm, wr), (by, bm, br) = ref.layer_norm(x, w, b, eps)
    ref.check(mean, wm, bm + ref.TINY[torch.float32], "mean")
    ref.check(rstd, wr, br, "rstd")
    ref.check(y, wy, ref.rounded(by, wy, x.dtype), "y")


def backward(sar, dy, x, w, mean, rstd, wdtype, gap=0, offset=0, params=True):
    rows, cols = x.shape
    dyv, _ = placed(dy, gap, offset)
    xv, _ = placed(x, gap, offset)
    dxv, dxf = placed(torch.zeros_like(x), gap, offset)
    dw = torch.full((cols,), MARK, dtype=wdtype, device="cuda") if params else None
    db = torch.full((cols,), MARK, dtype=wdtype, device="cuda") if params else None
    need = sar.sar_layer_norm_backward_workspace_bytes(rows, cols)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN all over
    sar.sar_layer_norm_backward(dyv, xv, w, mean, rstd, dxv, dw, db, workspace=ws[:need] if params else None)
    torch.cuda.synchronize()
    assert untouched(dxv, dxf) and bool((ws[need:] == 0xFF).all())
    return dxv, dw, db


def check_backward(sar, dy, x, w, wdtype, gap=0, offset=0):
    _, mean, rstd = (t.float() for t in ref.layer_norm(x, None, None, 1e-5)[0])
    dx, dw, db = backward(sar, dy, x, w, mean, rstd, wdtype, gap, offset)
    (wx, ww, wb), (bx, bw, bb) = ref.layer_norm_backward(dy, x, w, mean, rstd)
    ref.check(dx, wx, ref.rounded(bx, wx, x.dtype), "dx")
    ref.check(dw, ww, ref.rounded(bw, ww, wdtype), "dweight")
    ref.check(db, wb, ref.rounded(bb, wb, wdtype), "dbias")


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (33, 64), (4, 257), (7, 511), (9, 1024), (130, 1021), (3, 2048), (5, 4096),
          (2, 4104), (3, 8192), (2, 16384), (1, 20000), (2, 33000), (1, 65536), (2, 140001), (700, 96), (2049, 40)]
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")]


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(sar, shape, types):
    dt, wt = (ref.DTYPES[t] for t in types)
    x, _, w, b = inputs(*shape, dt, wt)
    check_forward(sar, x, w, b)


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(sar, shape, types):
    dt, wt = (ref.DTYPES[t] for t in types)
    x, dy, w, _ = inputs(*shape, dt, wt)
    check_backward(sar, dy, x, w, wt)


# Rows enough to stay in the blocks for long, at every split of a row over threads, whole and partly filled.
MANY = [(2500, 4096), (2443, 4090), (330, 8192), (333, 5004), (320, 16384), (306, 12290), (4900, 2048), (9800, 1024), (9740, 520),
        (18300, 512), (18250, 300), (39000, 256), (38950, 132), (20011, 64), (6100, 1150), (305, 4096), (1217, 1024)]


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_rows(sar, shape, types):
    dt, wt = (ref.DTYPES[t] for t in types)
    x, dy, w, b = inputs(*shape, dt, wt, seed=shape[0])
    check_forward(sar, x, w, b)
    check_backward(sar, dy, x, w, wt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gap,offset", [(8, 8), (2, 4), (1, 0), (0, 1)])
@pytest.mark.parametrize("shape", [(9740, 1000), (4870, 2048), (600, 9000), (18300, 400)], ids=str)
def test_many_rows_strides_and_alignment(sar, shape, gap, offset, dtype):
    dt = ref.DTYPES[dtype]
    x, dy, w, b = inputs(*shape, dt, dt, seed=1)
    check_forward(sar, x, w, b, gap=gap, offset=offset)
    check_backward(sar, dy, x, w, dt, gap=gap, offset=offset)


@pytest.mark.parametrize("shape", [(700, 4096), (5000, 1021), (320, 9001)], ids=str)
def test_many_rows_without_parameters_in_place(sar, shape):
    """No weight or bias, statistics not wanted, y over x and dx over dy; a NaN row stays alone."""
    x, dy, _, _ = inputs(*shape, torch.float32, torch.float32, seed=2)
    x[5, 7] = float("nan")
    (wy, mean, rstd), (by, _, _) = ref.layer_norm(x, None, None, 1e-5)
    y = x.clone()
    sar.sar_layer_norm(y, y)
    assert bool(torch.isnan(y[5]).all())
    ref.check(y, torch.where(torch.isnan(wy), float("nan"), wy), ref.rounded(by, wy, x.dtype), "y")
    mean, rstd = mean.float(), rstd.float()
    (wx, _, _), (bx, _, _) = ref.layer_norm_backward(dy, x, None, mean, rstd)
    sar.sar_layer_norm_backward(dy, x, None, mean, rstd, dy)
    ref.check(dy, wx, ref.rounded(bx, wx, x.dtype), "dx")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gap,offset", [(0, 1), (8, 0), (5, 0), (16, 8), (3, 2), (1, 16)])
@pytest.mark.parametrize("shape", [(6, 100), (5, 1024), (3, 4096), (3, 9000)], ids=str)
def test_strides_and_alignment(sar, shape, gap, offset, dtype):
    dt = ref.DTYPES[dtype]
    x, dy, w, b = inputs(*shape, dt, dt, seed=1)
    check_forward(sar, x, w, b, gap=gap, offset=offset)
    check_backward(sar, dy, x, w, dt, gap=gap, offset=offset)


@pytest.mark.parametrize("cols", [100, 1024, 4096])
def test_layouts_of_their_own(sar, cols):
    """x, dy and the outputs each with another leading dimension and alignment; parameters off 16 bytes."""
    x, dy, w, b = inputs(9, cols, torch.bfloat16, torch.float32, seed=2)
    wv, bv = (torch.cat([t[:1], t])[1:] for t in (w, b))
    assert wv.data_ptr() % 16 != 0
    xv, _ = placed(x, 8, 0)
    dyv, _ = placed(dy, 3, 1)
    yv, yf = placed(torch.zeros_like(x), 0, 0)
    sar.sar_layer_norm(xv, yv, wv, bv)
    (wy, mean, rstd), (by, _, _) = ref.layer_norm(x, w, b, 1e-5)
    ref.check(yv, wy, ref.rounded(by, wy, x.dtype), "y")
    assert untouched(yv, yf)
    dxv, dxf = placed(torch.zeros_like(x), 24, 16)
    mean, rstd = mean.float(), rstd.float()
    dw = torch.zeros(cols + 1, device="cuda")[1:]
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(9, cols), dtype=torch.uint8, device="cuda")
    sar.sar_layer_norm_backward(dyv, xv, wv, mean, rstd, dxv, dw, None, workspace=ws)
    (wx, ww, _), (bx, bw, _) = ref.layer_norm_backward(dy, x, w, mean, rstd)
    ref.check(dxv, wx, ref.rounded(bx, wx, x.dtype), "dx")
    ref.check(dw, ww, ref.rounded(bw, ww, torch.float32), "dweight")
    assert untouched(dxv, dxf)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cols", [77, 1024, 5000])
def test_optional_arguments(sar, cols, dtype):
    dt = ref.DTYPES[dtype]
    x, dy, w, b = inputs(4, cols, dt, dt, seed=3)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y = torch.empty_like(x)
        sar.sar_layer_norm(x, y, ww, bb)
        (wy, mean, rstd), (by, _, _) = ref.layer_norm(x, ww, bb, 1e-5)
        ref.check(y, wy, ref.rounded(by, wy, dt), "y")
    mean, rstd = mean.float(), rstd.float()
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(4, cols), dtype=torch.uint8, device="cuda")
    (wx, wdw, wdb), (bx, bdw, bdb) = ref.layer_norm_backward(dy, x, None, mean, rstd)
    for has_w, has_b in ((True, False), (False, True), (False, False)):
        dx = torch.empty_like(x)
        dw = torch.empty_like(w) if has_w else None
        db = torch.empty_like(b) if has_b else None
        sar.sar_layer_norm_backward(dy, x, None, mean, rstd, dx, dw, db, workspace=ws if has_w or has_b else None)
        ref.check(dx, wx, ref.rounded(bx, wx, dt), "dx")
        if has_w:
            ref.check(dw, wdw, ref.rounded(bdw, wdw, dt), "dweight")
        if has_b:
            ref.check(db, wdb, ref.rounded(bdb, wdb, dt), "dbias")


@pytest.mark.parametrize("cols", [64, 1000, 4096, 70000])
def test_in_place(sar, cols):
    x, dy, w, b = inputs(5, cols, torch.bfloat16, torch.bfloat16, seed=4)
    y, mean, rstd = forward(sar, x, w, b)
    z = x.clone()
    sar.sar_layer_norm(z, z, w, b)
    assert torch.equal(z, y)
    dx, dw, db = backward(sar, dy, x, w, mean, rstd, torch.bfloat16)
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(5, cols), dtype=torch.uint8, device="cuda")
    for which in ("dy", "x"):
        a, c = dy.clone(), x.clone()
        into = a if which == "dy" else c
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        sar.sar_layer_norm_backward(a, c, w, mean, rstd, into, dw2, db2, workspace=ws)
        assert torch.equal(into, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("cols", [48, 1024, 3000, 40000])
def test_no_rows_and_no_columns(sar, cols):
    x = torch.empty(0, cols, device="cuda")
    sar.sar_layer_norm(x, torch.empty_like(x))
    dw, db = torch.full((cols,), MARK, device="cuda"), torch.full((cols,), MARK, device="cuda")
    ws = torch.full((sar.sar_layer_norm_backward_workspace_bytes(0, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    e = torch.empty(0, device="cuda")
    sar.sar_layer_norm_backward(x, x, None, e, e, torch.empty_like(x), dw, db, workspace=ws)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    z = torch.empty(3, 0, device="cuda")
    sar.sar_layer_norm(z, torch.empty_like(z))


@pytest.mark.parametrize("cols", [40, 1024, 4096, 50000])
def test_rows_without_spread_and_far_from_zero(sar, cols):
    """Constant rows (variance 0, so rstd = 1 / sqrt(eps)), and rows whose mean is 1000 times their spread: the
    deviations' variance keeps its digits, where the squares' sum would not."""
    x = torch.full((3, cols), 2.5, device="cuda")
    x[1] = 0.0
    x[2] = -7.0
    check_forward(sar, x, None, None, eps=1e-3)
    check_forward(sar, *inputs(4, cols, torch.float32, torch.float32, seed=5, spread=0.01, shift=10.0)[::2], None, eps=1e-12)


@pytest.mark.parametrize("cols", [33, 1024, 4100])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_infinities_and_nan_stay_in_their_rows(sar, cols, dtype):
    dt = ref.DTYPES[dtype]
    x, dy, w, b = inputs(6, cols, dt, dt, seed=6)
    x[1, cols // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4, cols - 1] = torch.finfo(dt).max if dtype != "fp32" else 1e18
    y, mean, rstd = forward(sar, x, w, b)
    for r in (1, 3):
        assert bool(torch.isnan(y[r]).all())
    keep = [0, 2, 5] if dtype == "bf16" else [0, 2, 4, 5]        # bf16's largest value overflows the squares
    (wy, _, _), (by, _, _) = ref.layer_norm(x[keep], w, b, 1e-5)
    ref.check(y[keep], wy, ref.rounded(by, wy, dt), "y")
    _, mean, rstd = (t.float() for t in ref.layer_norm(x, None, None, 1e-5)[0])
    dx, _, _ = backward(sar, dy, x, w, mean, rstd, dt)
    clean = [0, 2, 5]
    (wx, _, _), (bx, _, _) = ref.layer_norm_backward(dy[clean], x[clean], w, mean[clean], rstd[clean])
    ref.check(dx[clean], wx, ref.rounded(bx, wx, dt), "dx")
    assert bool(torch.isnan(dx[3]).all())


@pytest.mark.parametrize("cols", [50, 1024])
def test_gradient_against_differences(sar, cols):
    """Differences of the forward kernel along a direction against the backward kernel's gradient.  With L = sum(y * dy):
    a difference is off by the forward bound of each y, weighted with dy, over the step; what the step's length itself
    costs is measured on the 64-bit formula."""
    rows, step = 6, 2.0 ** -5
    x, dy, w, b = inputs(rows, cols, torch.float32, torch.float32, seed=7)
    g = torch.Generator(device="cuda").manual_seed(8)
    along = {"x": torch.randn(rows, cols, generator=g, device="cuda"), "w": torch.randn(cols, generator=g, device="cuda"),
             "b": torch.randn(cols, generator=g, device="cuda")}
    _, mean, rstd = forward(sar, x, w, b)
    dx, dw, db = backward(sar, dy, x, w, mean, rstd, torch.float32)
    (ex, ew, eb), bounds = ref.layer_norm_backward(dy, x, w, *(t.float() for t in ref.layer_norm(x, w, b, 1e-5)[0][1:]))
    for name, grad, exact, bound in (("x", dx, ex, bounds[0]), ("w", dw, ew, bounds[1]), ("b", db, eb, bounds[2])):
        ends, true_ends, room = [], [], 0.0
        for sign in (1, -1):
            p = {"x": x, "w": w, "b": b}
            p[name] = p[name] + sign * step * along[name]
            y = forward(sar, p["x"], p["w"], p["b"])[0]
            (ty, _, _), (by, _, _) = ref.layer_norm(p["x"], p["w"], p["b"], 1e-5)
            ends.append((y.double() * dy.double()).sum().item())
            true_ends.append((ty * dy.double()).sum().item())
            room += ((ref.rounded(by, ty, torch.float32)) * dy.double().abs()).sum().item()
        slope, true_slope = ((e[0] - e[1]) / (2 * step) for e in (ends, true_ends))
        d = along[name].double()
        own, truth = (grad.double() * d).sum().item(), (exact * d).sum().item()
        allowed = abs(true_slope - truth) + room / (2 * step) + ((bound + ref.U * exact.abs()) * d.abs()).sum().item()
        assert abs(slope - own) <= allowed, (name, slope, own, allowed)
        assert allowed < 0.05 * (abs(truth) + (exact.abs() * d.abs()).sum().item() ** 0.5)     # the check says something


@pytest.mark.parametrize("shape", [(8, 4096), (515, 1024), (300, 1021), (70, 12000), (4900, 2048), (5000, 1021)], ids=str)
def test_same_bits_on_every_run_and_stream(sar, shape):
    x, dy, w, b = inputs(*shape, torch.bfloat16, torch.float32, seed=9)
    y, mean, rstd = forward(sar, x, w, b)
    first = backward(sar, dy, x, w, mean, rstd, torch.float32)
    side = torch.cuda.Stream()
    for s in (None, side):
        if s is not None:
            s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y2 = torch.empty_like(x)
            sar.sar_layer_norm(x, y2, w, b)
            dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
            ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(*shape), dtype=torch.uint8, device="cuda")
            sar.sar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(y2, y)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), first))


def test_captured_in_a_graph(sar):
    x, dy, w, b = inputs(64, 2048, torch.float16, torch.float32, seed=10)
    y, mean, rstd = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(64, 2048), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sar.sar_layer_norm(x, y, w, b, mean, rstd)
        sar.sar_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws)
    x2, dy2, _, _ = inputs(64, 2048, torch.float16, torch.float32, seed=11)
    x.copy_(x2)
    dy.copy_(dy2)
    graph.replay()
    torch.cuda.synchronize()
    y3, mean3, rstd3 = forward(sar, x2, w, b)
    want = backward(sar, dy2, x2, w, mean3, rstd3, torch.float32)
    assert torch.equal(y, y3) and all(torch.equal(p, q) for p, q in zip((dx, dw, db), want))


def test_offsets_past_32_bits(sar):
    """Two rows over 2^31 elements apart."""
    ld = 2 ** 31 + 24
    flat = torch.empty(ld + 1000, dtype=torch.bfloat16, device="cuda")
    x, dy, w, b = inputs(2, 1000, torch.bfloat16, torch.float32, seed=12)
    far = torch.as_strided(flat, (2, 1000), (ld, 1))
    far.copy_(x)
    y, mean, rstd = forward(sar, x, w, b)
    sar.sar_layer_norm(far, far, w, b)
    assert torch.equal(far, y)
    far.copy_(x)
    want = backward(sar, dy, x, w, mean, rstd, torch.float32)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(sar.sar_layer_norm_backward_workspace_bytes(2, 1000), dtype=torch.uint8, device="cuda")
    sar.sar_layer_norm_backward(dy, far, w, mean, rstd, far, dw, db, workspace=ws)
    assert torch.equal(far, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, want[2])
