"""cr_rmsnorm and cr_rmsnorm_backward against the FP64 oracle.

Tolerances.  A sum of n FP32 terms errs by at most n 2^-24 of the sum of magnitudes, so the norm's
relative error is d = (D + 32) 2^-24 (half of it from the root, the rest for the few operations
around it); outputs are rounded once to their type."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import ROUND, TYPES, matrix, values, vector, within

pytestmark = pytest.mark.gpu
SIZES = [(1, 1), (3, 7), (32, 5), (100, 33), (256, 64), (1000, 17), (1024, 3), (2560, 9), (4096, 130), (8192, 2), (12345, 3),
         (20000, 2)]


def _inputs(D, T, kind, residual, pad=0, shift=0, seed=0):
    rng = np.random.default_rng(seed + D + T)
    X = matrix(rng.normal(size=(D, T)) * 2, TYPES[kind], pad, shift)
    R = matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift) if residual else None
    return rng, X, R, np.float32(1 + 0.2 * rng.normal(size=D))


def _check(lib, D, T, kind, residual, e4m3, pad=0, shift=0, eps=1e-5):
    _, X, R, g = _inputs(D, T, kind, residual, pad, shift)
    y, h = trend.rmsnorm(values(X), g.astype(float), values(R) if residual else None, eps)
    d = (D + 32) * 2.0 ** -24
    if e4m3:
        Y, scale, H = lib.rmsnorm_e4m3(X, vector(g), R, eps=eps)
        s = trend.column_scale(y)
        within(scale, s, d * s, torch.float32)
        within(Y, y / s, 3 * d * np.abs(y / s), torch.float8_e4m3fn)
        assert np.abs(values(Y)).max() <= 448
    else:
        Y, H = lib.rmsnorm(X, vector(g), R, eps=eps)
        within(Y, y, d * np.abs(y), TYPES[kind])
    if residual:
        within(H, h, 2.0 ** -24 * np.abs(h), TYPES[kind])
    else:
        assert H is None


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,T", SIZES)
def test_rmsnorm(lib, kind, D, T):
    for residual in (False, True):
        for e4m3 in (False, True):
            _check(lib, D, T, kind, residual, e4m3)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (16, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rmsnorm_strides(lib, kind, pad, shift):
    for D in (48, 1000, 4096):
        _check(lib, D, 6, kind, True, True, pad, shift)
        _check(lib, D, 6, kind, False, False, pad, shift)


def test_rmsnorm_many_columns(lib):
    _check(lib, 64, 70000, "bf16", True, True)
    _check(lib, 768, 3001, "f16", True, False)


def test_rmsnorm_special_columns(lib):
    """All-zero, NaN, infinite and tiny columns beside an ordinary one: none touches another."""
    for D in (40, 1500, 6000):
        x = np.random.default_rng(1).normal(size=(D, 6))
        x[:, 0] = 0
        x[D // 2, 1] = np.nan
        x[D - 1, 2] = np.inf
        x[:, 3] *= 1e-30
        g = vector(np.ones(D))
        X = matrix(x, torch.float32)
        Y, scale, _ = lib.rmsnorm_e4m3(X, g, eps=1e-6)
        Y, s = values(Y), values(scale)
        assert (Y[:, 0] == 0).all() and s[0] == np.float32(2.0 ** -100) / np.float32(448)
        assert np.isnan(Y[:, 1]).all() and np.isnan(s[1]) and np.isnan(Y[:, 2]).all() and np.isnan(s[2])
        assert np.isfinite(Y[:, 3:]).all()
        ref, refs, _ = lib.rmsnorm_e4m3(X[:, 4:], g, eps=1e-6)
        np.testing.assert_array_equal(Y[:, 4:], values(ref))
        np.testing.assert_array_equal(s[4:], values(refs))
        zero = values(lib.rmsnorm(X[:, :1], g, eps=0.0)[0])   # 0 / 0
        assert np.isnan(zero).all()


def test_rmsnorm_in_place_residual_and_streams(lib):
    _, X, R, g = _inputs(640, 50, "bf16", True)
    want, H = lib.rmsnorm(X, vector(g), R)
    gv = vector(g)
    Y = torch.empty(50, 640, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    lib._check(lib._lib.cr_rmsnorm(2, X.data_ptr(), 640, R.data_ptr(), 640, gv.data_ptr(), 640, 50, 1e-6, R.data_ptr(), 640, 2,
                                   Y.data_ptr(), 640, None, st))
    assert torch.equal(Y.T, want) and torch.equal(R, H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, _ = lib.rmsnorm(X, gv, stream=s)
    s.synchronize()
    assert torch.equal(a, lib.rmsnorm(X, gv)[0])
    assert lib.rmsnorm(X[:, :0], gv)[0].shape == (640, 0)


def _backward(lib, D, T, kind, dh, pad=0, shift=0, eps=1e-5):
    rng, X, _, g = _inputs(D, T, kind, False, pad, shift)
    dY = matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift)
    dH = matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift) if dh else None
    dX, dg = lib.rmsnorm_backward(X, vector(g), dY, dH, eps=eps)
    h, dy, gv = values(X), values(dY), g.astype(float)
    oX, og = trend.rmsnorm_backward(h, gv, dy, values(dH) if dh else None, eps)
    r = 1 / np.sqrt(np.mean(h * h, axis=0) + eps)
    u = gv[:, None] * dy
    d = (D + 64) * 2.0 ** -23
    err = d * (np.abs(r * u) + np.abs(h) * r ** 3 * np.mean(np.abs(u * h), axis=0)) + 2.0 ** -22 * np.abs(oX)
    within(dX, oX, err, TYPES[kind])
    within(dg, og, (T + D + 64) * 2.0 ** -23 * np.sum(np.abs(dy * h * r), axis=1), torch.float32)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,T", SIZES + [(64, 5000), (777, 1003)])
def test_rmsnorm_backward(lib, kind, D, T):
    _backward(lib, D, T, kind, False)
    _backward(lib, D, T, kind, True)


def test_rmsnorm_backward_long_columns(lib):
    """Columns too long for registers, enough of them for the gradient of gamma to be summed in parts."""
    _backward(lib, 17001, 70, "bf16", True)
    _backward(lib, 16400, 37, "f32", False)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1)])
def test_rmsnorm_backward_strides(lib, pad, shift):
    for D in (48, 1000, 4096):
        _backward(lib, D, 37, "bf16", True, pad, shift)


def test_rmsnorm_backward_parts_in_place_and_empty(lib):
    rng, X, _, g = _inputs(520, 300, "f16", False)
    dY, dH = matrix(rng.normal(size=(520, 300)), torch.float16), matrix(rng.normal(size=(520, 300)), torch.float16)
    gv = vector(g)
    dX, dg = lib.rmsnorm_backward(X, gv, dY, dH)
    for _ in range(3):
        again = lib.rmsnorm_backward(X, gv, dY, dH)
        assert torch.equal(again[0], dX) and torch.equal(again[1], dg)
    st = torch.cuda.current_stream().cuda_stream
    only = torch.empty(520, device="cuda")
    lib._check(lib._lib.cr_rmsnorm_backward(1, X.data_ptr(), 520, gv.data_ptr(), dY.data_ptr(), 520, None, 0, 520, 300, 1e-6, None,
                                            0, only.data_ptr(), st))
    assert torch.equal(only, dg)
    place = dY.T.contiguous().T
    lib._check(lib._lib.cr_rmsnorm_backward(1, X.data_ptr(), 520, gv.data_ptr(), place.data_ptr(), 520, dH.data_ptr(), 520, 520, 300,
                                            1e-6, place.data_ptr(), 520, only.data_ptr(), st))
    assert torch.equal(place, dX) and torch.equal(only, dg)
    _, none = lib.rmsnorm_backward(X[:, :0], gv, dY[:, :0])
    assert not none.any()


def test_rmsnorm_gradient_against_differences(lib):
    """FP32, one direction: |f''| h^2 and FP32 sums of about 1e-6 / h of f, both below 1 % at 2^-7."""
    rng, X, _, g = _inputs(96, 40, "f32", False)
    dY = matrix(rng.normal(size=(96, 40)), torch.float32)
    D = matrix(rng.normal(size=(96, 40)), torch.float32)
    gv, h = vector(g), 2.0 ** -7
    f = lambda x: float((lib.rmsnorm(x, gv)[0].double() * dY.double()).sum())   # noqa: E731
    dX, _ = lib.rmsnorm_backward(X, gv, dY)
    slope = float((dX.double() * D.double()).sum())
    diff = (f(X + h * D) - f(X - h * D)) / (2 * h)
    assert abs(slope - diff) <= 0.01 * max(abs(slope), float(dX.norm()))


def test_rmsnorm_binding_refusals(lib):
    x, g = torch.zeros(8, 4, device="cuda").half(), torch.ones(8, device="cuda")
    for call in (lambda: lib.rmsnorm(x, g[:7]), lambda: lib.rmsnorm(x, g.half()), lambda: lib.rmsnorm(x, g, x.float()),
                 lambda: lib.rmsnorm(x, g, x[:, :3]), lambda: lib.rmsnorm(x.to(torch.float8_e4m3fn), g),
                 lambda: lib.rmsnorm(x, g, eps=-1.0), lambda: lib.rmsnorm_backward(x, g, x.float()),
                 lambda: lib.rmsnorm(x.double(), g)):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
    assert ROUND
