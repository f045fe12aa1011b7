"""Refusals of the operators around the allreduce, without a GPU: every
argument error comes back before anything is launched."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


A, B, C, D = 1 << 20, 2 << 20, 3 << 20, 4 << 20
BF16, FP16, FP32, E4M3 = 0, 1, 2, 3
HUGE = 2 ** 61


def test_layer_norm_refusals(sar):
    def call(x=A, ldx=64, w=None, b=None, y=B, ldy=64, mean=None, rstd=None, rows=4, cols=64, eps=1e-5, dt=BF16, wdt=FP32):
        return sar.lib.sar_layer_norm(x, ldx, w, b, y, ldy, mean, rstd, rows, cols, ctypes.c_float(eps), dt, wdt, None)
    for dt, wdt in ((E4M3, E4M3), (4, FP32), (7, FP32), (BF16, FP16), (FP32, BF16), (FP16, E4M3), (BF16, 9)):
        assert call(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(x=None), dict(y=None), dict(ldx=63), dict(ldy=63), dict(eps=-1e-9), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(rows=HUGE), dict(ldx=HUGE, rows=9)):
        assert call(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(x=A + 1), dict(y=B + 1), dict(w=C + 2), dict(b=C + 1), dict(mean=C + 2), dict(rstd=C + 1)):
        assert call(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert call(w=C + 1, wdt=BF16) == sar.SAR_ERR_MISALIGNED
    assert call(x=None, y=None, rows=0) == sar.SAR_OK
    assert call(x=None, y=None, cols=0) == sar.SAR_OK


def test_layer_norm_backward_refusals(sar):
    need = sar.sar_layer_norm_backward_workspace_bytes(4, 64)
    assert need >= 16

    def call(dy=A, lddy=64, x=B, ldx=64, w=None, mean=C, rstd=C, dx=D, lddx=64, dw=C, db=C, rows=4, cols=64, dt=BF16,
             wdt=FP32, ws=D, n=need):
        return sar.lib.sar_layer_norm_backward(dy, lddy, x, ldx, w, mean, rstd, dx, lddx, dw, db, rows, cols, dt, wdt, ws,
                                               n, None)
    for dt, wdt in ((E4M3, FP32), (BF16, FP16), (FP32, FP16)):
        assert call(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(lddy=3), dict(ldx=3),
               dict(lddx=3), dict(ws=None), dict(n=need - 1), dict(rows=HUGE), dict(ws=None, dw=None), dict(ws=None, db=None)):
        assert call(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(dy=A + 1), dict(x=B + 1), dict(dx=D + 1), dict(mean=C + 2), dict(rstd=C + 2), dict(dw=C + 2),
               dict(db=C + 2), dict(w=C + 2), dict(ws=D + 8)):
        assert call(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert call(cols=0) == sar.SAR_OK
    assert call(rows=0, dw=None, db=None, ws=None) == sar.SAR_OK
    assert call(rows=0, ws=None) == sar.SAR_ERR_INVALID_ARG
    assert sar.sar_layer_norm_backward_workspace_bytes(4, HUGE) == 0


def test_expert_sort_refusals(sar):
    def call(ids=A, size=8, tokens=4, topk=2, experts=8, align=1, cap=8, counts=B, offsets=B, pos=C, src=D):
        return sar.lib.sar_expert_sort(ids, size, tokens, topk, experts, align, cap, counts, offsets, pos, src, None)
    for kw in (dict(size=2), dict(size=0), dict(topk=0), dict(topk=-1), dict(experts=0), dict(experts=1025), dict(align=0),
               dict(tokens=2 ** 31), dict(tokens=2 ** 30, topk=2), dict(tokens=HUGE), dict(cap=2 ** 31), dict(align=2 ** 30),
               dict(ids=None), dict(counts=None), dict(offsets=None), dict(pos=None)):
        assert call(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(ids=A + 4), dict(ids=A + 2, size=4), dict(counts=B + 1), dict(offsets=B + 2), dict(pos=C + 2), dict(src=D + 3)):
        assert call(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert sar.sar_expert_rows(10, 2, 4, 16) == 20 + 4 * 15
    assert sar.sar_expert_rows(1, 2, 100, 128) == 2 + 2 * 127
    assert sar.sar_expert_rows(0, 2, 100, 128) == 0
    for bad in ((10, 0, 4, 1), (10, 2, 0, 1), (10, 2, 1025, 1), (10, 2, 4, 0), (2 ** 31, 1, 4, 1)):
        assert sar.sar_expert_rows(*bad) == 0


def test_expert_dispatch_and_combine_refusals(sar):
    def dispatch(x=A, ldx=64, pos=B, counts=None, offsets=None, experts=8, rows=C, ldr=64, cap=8, tokens=4, topk=2, cols=64,
                 dt=BF16):
        return sar.lib.sar_expert_dispatch(x, ldx, pos, counts, offsets, experts, rows, ldr, cap, tokens, topk, cols, dt, None)
    assert dispatch(dt=5) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(x=None), dict(pos=None), dict(rows=None), dict(ldx=63), dict(ldr=63), dict(topk=0), dict(cap=2 ** 31),
               dict(counts=D), dict(offsets=D), dict(counts=D, offsets=D, experts=0), dict(tokens=2 ** 30), dict(ldr=HUGE)):
        assert dispatch(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(x=A + 1), dict(pos=B + 1), dict(rows=C + 1), dict(counts=D + 1, offsets=D)):
        assert dispatch(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert dispatch(tokens=0, x=None) == sar.SAR_OK
    assert dispatch(cols=0) == sar.SAR_OK
    assert dispatch(cap=0, rows=None) == sar.SAR_OK

    def combine(rows=A, ldr=64, cap=8, pos=B, w=None, out=C, ldo=64, tokens=4, topk=2, cols=64, dt=BF16, wdt=FP32):
        return sar.lib.sar_expert_combine(rows, ldr, cap, pos, w, out, ldo, tokens, topk, cols, dt, wdt, None)
    for dt, wdt in ((E4M3, FP32), (4, 4), (BF16, FP16), (FP32, BF16)):
        assert combine(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(rows=None), dict(pos=None), dict(out=None), dict(ldr=3), dict(ldo=3), dict(topk=0), dict(tokens=HUGE)):
        assert combine(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(rows=A + 1), dict(pos=B + 2), dict(out=C + 1), dict(w=D + 2)):
        assert combine(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert combine(tokens=0, out=None) == sar.SAR_OK

    def backward(dout=A, ldo=64, rows=B, ldr=64, cap=8, pos=C, w=D, counts=None, offsets=None, experts=8, drows=B, lddr=64,
                 dw=D, tokens=4, topk=2, cols=64, dt=BF16, wdt=FP32):
        return sar.lib.sar_expert_combine_backward(dout, ldo, rows, ldr, cap, pos, w, counts, offsets, experts, drows, lddr, dw,
                                                   tokens, topk, cols, dt, wdt, None)
    for dt, wdt in ((E4M3, FP32), (FP16, BF16)):
        assert backward(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(dout=None), dict(rows=None), dict(pos=None), dict(w=None), dict(drows=None), dict(ldo=3), dict(lddr=3),
               dict(ldr=3), dict(topk=0), dict(counts=D), dict(cap=2 ** 31)):
        assert backward(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(dout=A + 1), dict(rows=B + 1), dict(pos=C + 1), dict(w=D + 1), dict(drows=B + 1), dict(dw=D + 2)):
        assert backward(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert backward(tokens=0, dout=None, pos=None) == sar.SAR_OK


def test_binding_refuses_what_the_boundary_cannot_see(sar):
    x, f = torch.zeros(4, 8), torch.zeros(4)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: sar.sar_layer_norm(x, x), lambda: sar.sar_layer_norm(x, torch.zeros(4, 9)),
                 lambda: sar.sar_layer_norm(x.double(), x.double()), lambda: sar.sar_layer_norm(x[0], x[0]),
                 lambda: sar.sar_layer_norm_backward(x, x, None, f, f, torch.zeros(5, 8)),
                 lambda: sar.sar_layer_norm_backward(x, x, None, f, f, x),
                 lambda: sar.sar_expert_sort(i, f.int(), torch.zeros(5, dtype=torch.int32), i),
                 lambda: sar.sar_expert_dispatch(x, i, x), lambda: sar.sar_expert_dispatch(x, i[0], x),
                 lambda: sar.sar_expert_dispatch(x, i, x, dtype=0), lambda: sar.sar_expert_combine(x, i, x),
                 lambda: sar.sar_expert_combine(x, i, torch.zeros(4, 7)),
                 lambda: sar.sar_expert_combine_backward(x, x, i, f, x)):
        with pytest.raises(ValueError):
            call()


def test_binding_arguments(sar):
    import inspect
    assert list(inspect.signature(sar.sar_layer_norm).parameters) == ["x", "y", "weight", "bias", "mean", "rstd", "eps", "stream"]
    for call in (lambda: sar.sar_layer_norm(), lambda: sar.sar_layer_norm(torch.zeros(1, 1)),
                 lambda: sar.sar_layer_norm(1, 2, 3, 4, 5, 6, 7, 8, 9), lambda: sar.sar_layer_norm(1, 2, x=3),
                 lambda: sar.sar_layer_norm(1, 2, z=3)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        sar.sar_layer_norm(None, None)


def test_binding_lists_every_operator(sar):
    for name in ("sar_layer_norm", "sar_layer_norm_backward", "sar_layer_norm_backward_workspace_bytes", "sar_expert_rows",
                 "sar_expert_sort", "sar_expert_dispatch", "sar_expert_combine", "sar_expert_combine_backward"):
        assert callable(getattr(sar, name)) and name in open(sar.__file__).read().split('"""')[1] or "workspace" in name
