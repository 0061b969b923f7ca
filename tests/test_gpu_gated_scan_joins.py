"""Gated recurrence: what crosses the joins between the parts of a series (warps, chunks, groups).

A NaN or an infinity goes on to the end of its series however strongly the gates forget, products of
coefficients may leave FP32's range either way, and only a series' start cuts the past off.  Finite
values are held to the recurrence's error bound (test_gpu_gated_scan.py), others to their kind."""
import numpy as np
import pytest
import torch

from oracle import trend
from test_gpu_gated_scan import _check, _state_error
from trend_util import TYPES, matrix, values, within

pytestmark = pytest.mark.gpu


def _kind(a):
    """Finite values as 0, infinities as their sign, NaN as 2."""
    return np.where(np.isnan(a), 2.0, np.where(np.isinf(a), np.sign(a), 0.0))


def _offsets(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["coeff", "convex", "variance"])
@pytest.mark.parametrize("T", [3000, 65536])
def test_nonfinite_values_last_to_the_end_of_their_series(lib, kind, gate, T):
    rng = np.random.default_rng(T)
    D, off = 6, [0, 10, T - 40, T]
    g = rng.uniform(-0.99, 0.99, (D, T)) if gate == "coeff" else rng.normal(size=(D, T)) * 1.5 + 2
    x, dh, h0 = rng.normal(size=(D, T)), rng.normal(size=(D, T)), rng.normal(size=(D, 3))
    x[:3, 1000] = np.nan, np.inf, -np.inf
    dh[:3, T - 1000] = np.nan, np.inf, -np.inf
    h0[3:5, 1] = np.nan, np.inf
    G, X, dH, S = matrix(g, TYPES[kind]), matrix(x, TYPES[kind]), matrix(dh, TYPES[kind]), matrix(h0, torch.float32)
    H, hT, saved = lib.gated_scan(G, X, gate, _offsets(off), S, save=True)
    dG, dX, dh0 = lib.gated_scan_backward(G, X, dH, gate, _offsets(off), S, None, saved)
    with np.errstate(invalid="ignore"):
        Ho, To = trend.gated_scan(values(G), values(X), gate, off, values(S))
        oG, oX, o0 = trend.gated_scan_backward(values(G), values(X), values(dH), gate, off, values(S), np.zeros((D, 3)))
    assert np.isnan(Ho[0, 1000:T - 40]).all() and np.isfinite(Ho[:, T - 40:]).all()   # what is at stake
    np.testing.assert_array_equal(_kind(values(H)), _kind(Ho))
    np.testing.assert_array_equal(_kind(values(hT)), _kind(To))
    np.testing.assert_array_equal(_kind(values(dX)), _kind(oX))
    np.testing.assert_array_equal(_kind(values(dh0)), _kind(o0))
    rest = np.arange(T) != 1000   # there the coefficient gate's oracle has 0 * inf in x dc/dg
    np.testing.assert_array_equal(np.isfinite(values(dG))[:, rest], np.isfinite(oG)[:, rest])


@pytest.mark.parametrize("T", [300, 5000])
def test_coefficients_of_exactly_zero(lib, T):
    """0 h: nothing of a finite state, NaN of an infinite one."""
    rng = np.random.default_rng(1)
    D = 4
    g, x = rng.uniform(0.5, 0.9, (D, T)), rng.normal(size=(D, T))
    g[:, T // 2] = 0.0
    x[0, 50], x[1, 50] = np.nan, np.inf
    G, X = matrix(g, torch.float32), matrix(x, torch.float32)
    H, hT = lib.gated_scan(G, X, "coeff")
    with np.errstate(invalid="ignore"):
        Ho, To = trend.gated_scan(values(G), values(X), "coeff", [0, T], np.zeros((D, 1)))
    np.testing.assert_array_equal(_kind(values(H)), _kind(Ho))
    err, _ = _state_error(values(G)[2:], np.ones((2, T)), values(X)[2:], Ho[2:], [0, T], np.zeros((2, 1)))
    within(H[2:], Ho[2:], err, torch.float32)


def _finite(lib, g, x, dh, kind="f32"):
    """Forward and backward of one series against the oracle, all finite."""
    D, T = g.shape
    G, X, dH = matrix(g, TYPES[kind]), matrix(x, TYPES[kind]), matrix(dh, TYPES[kind])
    H, hT, saved = lib.gated_scan(G, X, "coeff", save=True)
    gv, xv, dv = values(G), values(X), values(dH)
    Ho, To = trend.gated_scan(gv, xv, "coeff", [0, T], np.zeros((D, 1)))
    err, _ = _state_error(gv, np.ones_like(gv), xv, Ho, [0, T], np.zeros((D, 1)))
    within(H, Ho, err, TYPES[kind])
    within(hT, To, err[:, -1:], torch.float32)
    _, dX, dh0 = lib.gated_scan_backward(G, X, dH, "coeff", None, None, None, saved)
    _, oX, o0 = trend.gated_scan_backward(gv, xv, dv, "coeff", [0, T], np.zeros((D, 1)), np.zeros((D, 1)))
    # q is the same recurrence run backwards: q_t = dh_t + a_{t+1} q_{t+1}
    ga = np.concatenate([np.zeros((D, 1)), gv[:, :0:-1]], axis=1)
    eq, _ = _state_error(ga, np.ones_like(gv), dv[:, ::-1], oX[:, ::-1], [0, T], np.zeros((D, 1)))
    within(dX, oX, eq[:, ::-1], TYPES[kind])
    within(dh0, o0, (np.abs(gv[:, 0]) * (eq[:, -1] + 2.0 ** -19 * np.abs(oX[:, 0])))[:, None], torch.float32)


@pytest.mark.parametrize("a,T", [(1.5, 2000), (-2.0, 700), (1.05, 9000), (300.0, 400)])
def test_growing_coefficients(lib, a, T):
    """A state that is zero for long, under coefficients whose products overflow: an impulse near the end, and
    for the gradients one near the start; one feature stays zero throughout."""
    D = 3
    late = max(1, min(40, int(60 / np.log2(abs(a)))))   # growth by at most 2^60
    x, dh = np.zeros((D, T)), np.zeros((D, T))
    x[0, T - late], x[1, T - 2] = 1.0, -3.0
    dh[0, late - 1], dh[1, 1] = 1.0, -3.0
    _finite(lib, np.full((D, T), a), x, dh)


def test_products_that_underflow_and_grow_again(lib):
    """Long runs of small coefficients before a few large ones: the past stays forgotten."""
    rng = np.random.default_rng(3)
    D, T = 5, 4000
    g = np.where(np.arange(T) % 500 < 488, 1e-3, 1e3) * rng.uniform(0.5, 1.0, (D, T))
    g[1] *= -1
    _finite(lib, g, rng.normal(size=(D, T)) * 1e-6, rng.normal(size=(D, T)) * 1e-6)


def test_groups_of_64_chunks(lib):
    """More than 1024 chunks in both directions."""
    _check(lib, 6, 140001, 1, "bf16", "convex")
    _check(lib, 3, 140001, 3, "f32", "coeff")


def test_underflow_and_growth_across_chunks(lib):
    """Whole chunks that forget everything, between chunks whose coefficients grow."""
    rng = np.random.default_rng(4)
    D, T = 4, 6000
    # 700 steps of 0.3, then 100 of 2 (a growth of 2^100 at most)
    g = np.where(np.arange(T) % 800 < 700, 0.3, 2.0) * np.ones((D, T))
    g[1] *= -1
    x, dh = rng.normal(size=(D, T)) * 1e-8, rng.normal(size=(D, T)) * 1e-8
    x[2, 100] += 1e4   # long gone before the first growth
    dh[2, T - 100] += 1e4
    _finite(lib, g, x, dh)
