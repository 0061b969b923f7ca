"""The FP64 statements of the trend-network operators against differences and closed forms, and
the refusals of the C entry points (CPU only: refused calls return before any device work)."""
import ctypes
import os

import numpy as np
import pytest

import mixed_precision_dense_mat_gb300 as cr
from mixed_precision_dense_mat_gb300 import build_lib
from oracle import trend

ACTS = ("none", "relu", "silu", "gelu")
GATES = ("coeff", "convex", "variance")


@pytest.fixture(scope="module")
def abi():
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    return cr.load()


def _differences(f, x, step=1e-6):
    """Central differences of the scalar f at every entry of x (error O(step^2))."""
    g = np.empty_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + step
        up = f()
        x[i] = old - step
        down = f()
        x[i] = old
        g[i] = (up - down) / (2 * step)
    return g


def _close(a, b):
    # differences: step^2 f''' / 6 + 2^-52 |f| / step, both below 1e-7 for these O(1)..O(10) values
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("act", ACTS)
def test_affine_gradient_against_differences(act):
    rng = np.random.default_rng(3)
    W, X, b, dY = rng.normal(size=(5, 4)), rng.normal(size=(5, 3)), rng.normal(size=4), rng.normal(size=(4, 3))
    f = lambda: float(np.sum(dY * trend.affine(W, X, b, act)[0]))   # noqa: E731
    dX, dW, db = trend.affine_backward(W, X, dY, trend.affine(W, X, b, act)[1], act)
    _close(dX, _differences(f, X))
    _close(dW, _differences(f, W))
    _close(db, _differences(f, b))


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(4)
    X, R, g = rng.normal(size=(6, 3)), rng.normal(size=(6, 3)), rng.normal(size=6)
    dY, dH = rng.normal(size=(6, 3)), rng.normal(size=(6, 3))

    def f():
        y, h = trend.rmsnorm(X, g, R, 0.01)
        return float(np.sum(dY * y) + np.sum(dH * h))

    dX, dg = trend.rmsnorm_backward(X + R, g, dY, dH, 0.01)
    _close(dX, _differences(f, X))
    _close(dX, _differences(f, R))
    _close(dg, _differences(f, g))


@pytest.mark.parametrize("gate", GATES)
def test_scan_gradient_against_differences(gate):
    rng = np.random.default_rng(5)
    off = [0, 3, 3, 4, 9]
    G, X = rng.normal(size=(2, 9)), rng.normal(size=(2, 9))
    h0, dH, dhT = rng.normal(size=(2, 4)), rng.normal(size=(2, 9)), rng.normal(size=(2, 4))

    def f():
        h, end = trend.gated_scan(G, X, gate, off, h0)
        return float(np.sum(dH * h) + np.sum(dhT * end))

    dG, dX, dh0 = trend.gated_scan_backward(G, X, dH, gate, off, h0, dhT)
    _close(dG, _differences(f, G))
    _close(dX, _differences(f, X))
    _close(dh0, _differences(f, h0))


def test_variance_gate_keeps_the_variance():
    g = np.linspace(-30, 30, 121)
    a, c, _, _ = trend.gate(g, "variance")
    np.testing.assert_allclose(a * a + c * c, 1.0, rtol=1e-12)


def _refused(code, *words):
    assert code == 1
    text = cr._lib.cr_last_error_detail().decode()
    for w in words:
        assert w in text, text


def test_affine_refusals(abi):
    p = 4096   # never read: every call below is refused first
    ok = dict(type=1, W=p, ldw=8, X=p, ldx=8, K=8, N=8, M=8, ws=None, xs=None, b=None, act=0, out=1, R=None, ldr=8, Z=None,
              ldz=8, Y=p, ldy=8, stream=None)

    def call(**kw):
        return cr._lib.cr_affine(*{**ok, **kw}.values())

    _refused(call(type=0), "type")
    _refused(call(type=7), "type")
    _refused(call(out=3), "out_type")
    _refused(call(act=4), "activation")
    _refused(call(act=-1), "activation")
    _refused(call(ws=p), "scales")
    _refused(call(K=0), "K >= 1")
    _refused(call(N=-3), "N >= 1")
    _refused(call(M=-1), "M >= 0")
    for ld in ("ldw", "ldx", "ldy"):
        _refused(call(**{ld: 7}), "leading dimension")
    _refused(call(R=p, ldr=7), "leading dimension")
    _refused(call(Z=p, ldz=7), "leading dimension")
    for null in ("W", "X", "Y"):
        _refused(call(**{null: None}), "NULL")
    assert call(M=0, X=None, Y=None) == 0   # nothing to do, no device call


def test_affine_backward_refusals(abi):
    p = 4096
    ok = dict(type=2, W=p, ldw=8, X=p, ldx=8, dY=p, lddy=8, Z=p, ldz=8, K=8, N=8, M=8, act=2, dX=p, lddx=8, dwt=2, dW=p,
              lddw=8, db=p, stream=None)

    def call(**kw):
        return cr._lib.cr_affine_backward(*{**ok, **kw}.values())

    _refused(call(type=3), "type")
    _refused(call(type=0), "type")
    _refused(call(act=9), "activation")
    _refused(call(dwt=1), "dw_type")
    _refused(call(K=0), "K >= 1")
    for null in ("W", "X", "dY", "Z"):
        _refused(call(**{null: None}), "NULL")
    for ld in ("ldw", "ldx", "lddy", "ldz", "lddx", "lddw"):
        _refused(call(**{ld: 7}), "leading dimension")


def test_rmsnorm_refusals(abi):
    p = 4096
    ok = dict(type=1, X=p, ldx=8, R=None, ldr=8, g=p, D=8, T=4, eps=1e-6, H=None, ldh=8, out=1, Y=p, ldy=8, s=None, stream=None)

    def call(**kw):
        return cr._lib.cr_rmsnorm(*{**ok, **kw}.values())

    _refused(call(type=3, out=3), "type")
    _refused(call(out=2), "out_type")
    _refused(call(out=3), "d_scale")
    _refused(call(s=p), "d_scale")
    _refused(call(D=0), "D >= 1")
    _refused(call(T=-1), "T >= 0")
    _refused(call(eps=-1.0), "eps")
    _refused(call(eps=float("nan")), "eps")
    _refused(call(ldx=7), "leading")
    _refused(call(H=p, ldh=7), "leading")
    for null in ("X", "g", "Y"):
        _refused(call(**{null: None}), "NULL")
    assert call(T=0, X=None, Y=None) == 0
    okb = dict(type=1, H=p, ldh=8, g=p, dY=p, lddy=8, dH=None, lddh=8, D=8, T=4, eps=1e-6, dX=p, lddx=8, dg=p, stream=None)

    def back(**kw):
        return cr._lib.cr_rmsnorm_backward(*{**okb, **kw}.values())

    _refused(back(type=3), "type")
    _refused(back(D=0), "D >= 1")
    _refused(back(eps=float("inf")), "eps")
    _refused(back(lddx=7), "leading")
    _refused(back(dH=p, lddh=7), "leading")
    for null in ("H", "g", "dY"):
        _refused(back(**{null: None}), "NULL")


def test_scan_refusals(abi):
    p = 4096
    ok = dict(type=1, gate=1, G=p, ldg=8, X=p, ldx=8, D=8, T=4, off=None, n=1, h0=None, ldh0=8, H=p, ldh=8, hT=None, ldhT=8,
              saved=None, stream=None)

    def call(**kw):
        return cr._lib.cr_gated_scan(*{**ok, **kw}.values())

    _refused(call(type=3), "type")
    _refused(call(gate=3), "gate")
    _refused(call(D=0), "D >= 1")
    _refused(call(T=-1), "T >= 0")
    _refused(call(n=2), "offsets")
    _refused(call(off=p, n=0), "series")
    _refused(call(off=p, n=-1), "n_seq")
    _refused(call(ldg=7), "leading")
    _refused(call(h0=p, ldh0=7), "leading")
    _refused(call(hT=p, ldhT=7), "leading")
    for null in ("G", "X"):
        _refused(call(**{null: None}), "NULL")
    okb = dict(type=1, gate=1, G=p, ldg=8, X=p, ldx=8, dH=p, lddh=8, D=8, T=4, off=None, n=1, h0=None, ldh0=8, dhT=None,
               lddhT=8, saved=p, dG=p, lddg=8, dX=p, lddx=8, dh0=None, lddh0=8, stream=None)

    def back(**kw):
        return cr._lib.cr_gated_scan_backward(*{**okb, **kw}.values())

    _refused(back(type=9), "type")
    _refused(back(gate=-1), "gate")
    _refused(back(n=3), "offsets")
    for ld in ("ldg", "ldx", "lddh", "lddg", "lddx"):
        _refused(back(**{ld: 7}), "leading")
    _refused(back(dh0=p, lddh0=7), "leading")
    for null in ("G", "X", "dH"):
        _refused(back(**{null: None}), "NULL")
    oks = dict(type=1, gate=1, G=p, ldg=8, X=p, ldx=8, h=p, ldh=8, D=8, B=2, H=None, ldo=8, hn=p, ldn=8, stream=None)

    def step(**kw):
        return cr._lib.cr_gated_step(*{**oks, **kw}.values())

    _refused(step(type=3), "type")
    _refused(step(gate=5), "gate")
    _refused(step(D=0), "D >= 1")
    _refused(step(B=-1), "B")
    _refused(step(ldn=7), "leading")
    for null in ("G", "X", "h", "hn"):
        _refused(step(**{null: None}), "NULL")
    assert step(B=0, G=None) == 0
    count = ctypes.c_size_t(7)
    assert cr._lib.cr_gated_scan_saved(3, 0, ctypes.byref(count)) == 0 and count.value == 0
    assert cr._lib.cr_gated_scan_saved(0, 5, ctypes.byref(count)) == 1
    assert cr._lib.cr_gated_scan_saved(3, 5, None) == 1
    assert cr._lib.cr_gated_scan_saved(2 ** 20, 2 ** 31 - 1, ctypes.byref(count)) == 0
    assert count.value > 2 ** 31   # counts pass 32 bits


def test_binding_constants():
    import re
    declared = {m.group(1): int(m.group(2))
                for m in re.finditer(r"\b(CR_[A-Z0-9_]+)\s*=\s*(\d+)", open(cr.HEADER).read())}
    for name in ("CR_TYPE_F32", "CR_TYPE_F16", "CR_TYPE_BF16", "CR_TYPE_E4M3", "CR_ACT_NONE", "CR_ACT_RELU", "CR_ACT_SILU",
                 "CR_ACT_GELU", "CR_GATE_COEFF", "CR_GATE_CONVEX", "CR_GATE_VARIANCE"):
        assert getattr(cr, name) == declared[name], name


def test_binding_refuses_host_tensors(abi):
    import torch
    x = torch.zeros(4, 4)
    for call in (lambda: cr.affine(x, x), lambda: cr.rmsnorm(x, x[0]), lambda: cr.gated_scan(x, x),
                 lambda: cr.gated_step(x, x, x)):
        with pytest.raises(cr.CrError) as e:
            call()
        assert e.value.code == 1
