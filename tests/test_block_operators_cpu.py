"""Refusals of the router, the expert layer and the orthogonalisation, without a
GPU: every argument error comes back before anything is launched."""
import ctypes
import inspect
import math

import pytest
import torch

A, B, C, D, E = (i << 20 for i in range(1, 6))
BF16, FP16, FP32, E4M3 = 0, 1, 2, 3
HUGE = 2 ** 61
NAMES = ["sar_expert_route", "sar_expert_route_backward", "sar_expert_layer", "sar_expert_layer_workspace_bytes",
         "sar_orthogonalize", "sar_orthogonalize_workspace_bytes"]


@pytest.fixture(scope="module")
def sar():
    import allreduce_reduction_rank_gb300 as s
    return s


@pytest.mark.parametrize("name", NAMES)
def test_the_package_lists(sar, name):
    assert callable(getattr(sar, name)) and name in dir(sar)
    assert f":func:`{name}`" in sar.__doc__


def test_route_refusals(sar):
    def call(x=A, ld=64, ids=B, size=4, w=C, tokens=4, topk=2, experts=64, softmax=0, dt=BF16, wdt=FP32):
        return sar.lib.sar_expert_route(x, ld, ids, size, w, tokens, topk, experts, softmax, dt, wdt, None)

    def backward(dw=C, x=A, ld=64, ids=B, size=4, dx=D, ldd=64, tokens=4, topk=2, experts=64, softmax=0, dt=BF16, wdt=FP32):
        return sar.lib.sar_expert_route_backward(dw, x, ld, ids, size, dx, ldd, tokens, topk, experts, softmax, dt, wdt, None)
    for f in (call, backward):
        for dt, wdt in ((E4M3, FP32), (BF16, FP16), (FP32, BF16), (9, FP32)):
            assert f(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
        for kw in (dict(x=None), dict(ids=None), dict(size=2), dict(topk=0), dict(topk=33, experts=64), dict(topk=3, experts=2, ld=2),
                   dict(experts=0, topk=1), dict(experts=1025, ld=1025), dict(ld=63), dict(softmax=2), dict(softmax=-1),
                   dict(tokens=2 ** 31), dict(tokens=HUGE), dict(ld=HUGE)):
            assert f(**kw) == sar.SAR_ERR_INVALID_ARG, kw
        for kw in (dict(x=A + 1), dict(ids=B + 2), dict(ids=B + 4, size=8)):
            assert f(**kw) == sar.SAR_ERR_MISALIGNED, kw
        assert f(tokens=0, x=None) == sar.SAR_OK
    assert call(w=None) == sar.SAR_ERR_INVALID_ARG and call(w=C + 2) == sar.SAR_ERR_MISALIGNED
    for kw in (dict(dw=None), dict(dx=None), dict(ldd=3)):
        assert backward(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    assert backward(dw=C + 2) == sar.SAR_ERR_MISALIGNED and backward(dx=D + 1) == sar.SAR_ERR_MISALIGNED


def test_layer_refusals(sar):
    size = sar.sar_expert_layer_workspace_bytes
    need = size(4, 2, 8, 64, 32)
    assert need >= 16
    for bad in ((4, 0, 8, 64, 32), (4, 2, 0, 64, 32), (4, 2, 1025, 64, 32), (513, 2, 8, 64, 32), (HUGE, 8, 8, 64, 32),
                (4, 2, 8, 2 ** 20 + 1, 32), (4, 2, 8, 64, 2 ** 20 + 1)):
        assert size(*bad) == 0
    assert size(512, 2, 8, 64, 32) > 0 and size(0, 2, 8, 64, 32) > 0 and size(4, 2, 8, 0, 0) > 0

    def call(x=A, ldx=64, ids=B, id_size=4, w=C, wi=D, wo=E, out=A, ldo=64, tokens=4, topk=2, experts=8, cols=64, hidden=32,
             gated=1, act=0, dt=BF16, wdt=FP32, ws=E, n=need):
        return sar.lib.sar_expert_layer(x, ldx, ids, id_size, w, wi, wo, out, ldo, tokens, topk, experts, cols, hidden, gated,
                                        act, dt, wdt, ws, n, None)
    for dt, wdt in ((E4M3, FP32), (BF16, FP16), (FP32, BF16), (9, FP32)):
        assert call(dt=dt, wdt=wdt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    for kw in (dict(x=None), dict(ids=None), dict(wi=None), dict(wo=None), dict(out=None), dict(ws=None), dict(n=need - 1),
               dict(id_size=3), dict(topk=0), dict(experts=0), dict(experts=1025), dict(tokens=513), dict(tokens=HUGE),
               dict(ldx=63), dict(ldo=63), dict(act=3), dict(act=-1), dict(cols=2 ** 20 + 1, ldx=HUGE), dict(hidden=2 ** 21)):
        assert call(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(x=A + 1), dict(ids=B + 2), dict(ids=B + 4, id_size=8), dict(w=C + 2), dict(wi=D + 1), dict(wo=E + 1),
               dict(out=A + 1), dict(ws=E + 8)):
        assert call(**kw) == sar.SAR_ERR_MISALIGNED, kw
    assert call(tokens=0, x=None) == sar.SAR_OK and call(cols=0, ldx=0, ldo=0, out=None) == sar.SAR_OK


def test_orthogonalize_refusals(sar):
    size = sar.sar_orthogonalize_workspace_bytes
    need = size(2, 64, 48)
    assert need >= 16
    for bad in ((65536, 4, 4), (1, 65537, 4), (1, 4, 65537), (HUGE, 4, 4)):
        assert size(*bad) == 0
    assert size(65535, 1, 1) > 0 and size(1, 65536, 65536) > 2 ** 32

    f = ctypes.c_float

    def call(g=A, ldg=48, gs=HUGE >> 10, out=B, ldo=48, os=1 << 20, batch=2, rows=64, cols=48, steps=5, a=3.4445, b=-4.775,
             c=2.0315, eps=1e-7, scale=1.0, dt=BF16, ws=E, n=need):
        return sar.lib.sar_orthogonalize(g, ldg, gs, out, ldo, os, batch, rows, cols, steps, f(a), f(b), f(c), f(eps), f(scale), dt,
                                         ws, n, None)
    for dt in (E4M3, 4, 9, -1):
        assert call(dt=dt) == sar.SAR_ERR_UNSUPPORTED_DTYPE
    inf, nan = math.inf, math.nan
    for kw in (dict(g=None), dict(out=None), dict(ws=None), dict(n=need - 1), dict(ldg=47), dict(ldo=47), dict(os=63 * 48 + 47),
               dict(gs=HUGE), dict(os=HUGE), dict(batch=65536), dict(rows=65537), dict(cols=65537, ldg=65537, ldo=65537),
               dict(steps=0), dict(steps=65), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf), dict(scale=nan), dict(scale=inf),
               dict(a=nan), dict(b=inf), dict(c=nan), dict(a=0.99), dict(a=0.0, b=1.0, c=0.0), dict(a=4.1), dict(a=2.0, b=0.0, c=0.0), dict(a=0.0, b=0.0, c=5.0),
               dict(a=1.0, b=8.0, c=-8.5)):
        assert call(**kw) == sar.SAR_ERR_INVALID_ARG, kw
    for kw in (dict(g=A + 1), dict(out=B + 1), dict(ws=E + 8)):
        assert call(**kw) == sar.SAR_ERR_MISALIGNED, kw
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert call(g=None, out=None, ws=None, **kw) == sar.SAR_OK, kw


def test_binding_refuses_what_the_boundary_cannot_see(sar):
    x, i, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    m = torch.zeros(2, 8, 8)
    for call in (lambda: sar.sar_expert_route(x, i, w), lambda: sar.sar_expert_route_backward(w, x, i, x),
                 lambda: sar.sar_expert_layer(x, i, m, m, x), lambda: sar.sar_orthogonalize(m, m, x),
                 lambda: sar.sar_expert_route(None, i, w), lambda: sar.sar_orthogonalize(x.double(), x.double(), x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sar.sar_expert_route(x, i), lambda: sar.sar_expert_layer(x, i, m, m), lambda: sar.sar_orthogonalize(m, m),
                 lambda: sar.sar_orthogonalize(m, m, x, step=3), lambda: sar.sar_expert_route(x, i, w, 0, None, 1)):
        with pytest.raises(TypeError):
            call()
    assert list(inspect.signature(sar.sar_orthogonalize).parameters) == [
        "g", "out", "workspace", "steps", "coefficients", "eps", "scale", "stream"]
