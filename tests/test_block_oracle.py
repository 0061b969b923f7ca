"""The FP64 statements of the gated product, the group norm and the orthogonalised update against differences and
closed forms, and the refusals of their C entries (CPU only: refused calls return before any device work)."""
import numpy as np
import pytest

import mixed_precision_dense_mat_gb300 as cr
from oracle import trend

ACTS = ("none", "relu", "silu", "gelu")
P = 4096   # never dereferenced: the calls end at their checks
F32, F16, BF16, E4M3 = 0, 1, 2, 3
BIG = 2 ** 31 - 1


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
def test_gated_gradient_against_differences(act):
    rng = np.random.default_rng(3)
    W, X, b, dY = rng.normal(size=(5, 8)), rng.normal(size=(5, 3)), rng.normal(size=8), rng.normal(size=(4, 3))
    f = lambda: float(np.sum(dY * trend.gated_affine(W, X, b, act)[0]))   # noqa: E731
    dX, dW, db = trend.gated_affine_backward(W, X, dY, trend.gated_affine(W, X, b, act)[1], act)
    _close(dX, _differences(f, X))
    _close(dW, _differences(f, W))
    _close(db, _differences(f, b))


@pytest.mark.parametrize("act", ACTS)
def test_group_norm_gradient_against_differences(act):
    rng = np.random.default_rng(4)
    X, dY = rng.normal(size=(6, 7)), rng.normal(size=(6, 7))
    gamma, beta, off = rng.normal(size=6), rng.normal(size=6), [0, 3, 3, 4, 7]
    f = lambda: float(np.sum(dY * trend.group_norm(X, 3, gamma, beta, act, off, 0.01)[0]))   # noqa: E731
    _, mean, rstd = trend.group_norm(X, 3, gamma, beta, act, off, 0.01)
    dX, dgamma, dbeta = trend.group_norm_backward(X, 3, gamma, beta, dY, mean, rstd, act, off)
    _close(dX, _differences(f, X))
    _close(dgamma, _differences(f, gamma))
    _close(dbeta, _differences(f, beta))


def test_group_norm_statistics():
    X = np.random.default_rng(5).normal(size=(8, 20)) + 3
    Y, mean, rstd = trend.group_norm(X, 2, np.ones(8), np.zeros(8), "none", [0, 20], 0.0)
    for g in range(2):
        y = Y[4 * g:4 * g + 4]
        assert abs(y.mean()) < 1e-14 and abs((y * y).mean() - 1) < 1e-14
        assert mean[g, 0] == X[4 * g:4 * g + 4].mean()


@pytest.mark.parametrize("K,N", [(5, 9), (9, 5), (6, 6), (1, 4), (1, 1)])
def test_orthogonalize_is_the_iteration(K, N):
    """The closed form by singular values against the products themselves."""
    G = np.random.default_rng(K + N).normal(size=(K, N))
    x = G / np.linalg.norm(G)
    a, b, c = 3.4445, -4.7750, 2.0315
    for _ in range(5):
        m = x @ x.T
        x = a * x + (b * m + c * m @ m) @ x
    np.testing.assert_allclose(trend.orthogonalize(G), x, rtol=1e-11, atol=1e-12)
    assert not trend.orthogonalize(np.zeros((K, N))).any()


def _refused(*calls):
    cr.load()
    for i, (f, args) in enumerate(calls):
        assert f(*args) == 1, i
        assert cr._lib.cr_last_error_detail(), i


def test_gated_refusals():
    L = cr.load()
    ok = [F16, P, 8, P, 8, 8, 4, 2, None, None, None, 2, F16, None, 0, P, 4, None]

    def but(i, v):
        return L.cr_gated_affine, [v if j == i else a for j, a in enumerate(ok)]

    _refused(but(0, F32), but(0, 9), but(2, 7), but(4, 7), but(5, 0), but(6, 0), but(7, -1), but(8, P), but(9, P), but(11, 4), but(11, -1),
             but(12, E4M3), but(1, None), but(3, None), but(15, None), but(16, 3))
    z = list(ok)
    z[13], z[14] = P, 7   # Z has 2 N rows
    _refused((L.cr_gated_affine, z))
    back = [F16, P, 8, P, 8, P, 4, P, 8, 8, 4, 2, 2, P, 8, F16, P, 8, P, None]

    def no(i, v):
        return L.cr_gated_affine_backward, [v if j == i else a for j, a in enumerate(back)]

    _refused(no(0, E4M3), no(0, F32), no(2, 7), no(4, 7), no(6, 3), no(8, 7), no(9, 0), no(10, 0), no(11, -1), no(12, 9), no(14, 7), no(15, BF16),
             no(17, 7), no(1, None), no(3, None), no(5, None), no(7, None))


def test_group_norm_refusals():
    L = cr.load()
    ok = [F16, P, 8, 8, 5, 2, P, 2, P, P, 1e-5, 2, P, 8, P, P, 2, None]

    def but(i, v):
        return L.cr_group_norm, [v if j == i else a for j, a in enumerate(ok)]

    _refused(but(0, E4M3), but(2, 7), but(3, 0), but(4, -1), but(5, 3), but(5, 0), but(5, 16), but(7, -1), but(10, -1.0), but(10, float("nan")),
             but(10, float("inf")), but(11, 4), but(13, 7), but(14, None), but(15, None), but(16, 1), but(1, None), but(12, None))
    back = [F16, P, 8, 8, 5, 2, P, 2, P, P, P, 8, P, P, 2, 2, P, 8, P, P, None]

    def no(i, v):
        return L.cr_group_norm_backward, [v if j == i else a for j, a in enumerate(back)]

    _refused(no(0, E4M3), no(2, 7), no(3, 0), no(4, -1), no(5, 3), no(7, -1), no(11, 7), no(14, 1), no(15, 4), no(17, 7), no(1, None),
             no(10, None), no(12, None), no(13, None))


def test_orthogonalize_refusals():
    L = cr.load()
    ok = [F32, P, 8, 8, 4, 5, 3.0, -4.0, 2.0, BF16, P, 8, None]

    def but(i, v):
        return L.cr_orthogonalize, [v if j == i else a for j, a in enumerate(ok)]

    _refused(but(0, E4M3), but(9, E4M3), but(1, None), but(10, None), but(2, 7), but(11, 7), but(3, 0), but(4, 0), but(5, 0), but(5, 101),
             but(6, float("nan")), but(7, float("inf")), but(8, 65.0))


def test_sizes_near_two_to_the_31_are_refused():
    L = cr.load()
    for big in (BIG, 2 ** 31 - 2 ** 16 + 1):
        calls = [(L.cr_gated_affine, [F16, P, BIG, P, BIG, *s, None, None, None, 2, F16, None, 0, P, BIG, None])
                 for s in ((big, 8, 8), (8, big, 8), (8, 8, big), (8, 2 ** 30, 8))]
        calls += [(L.cr_gated_affine_backward, [F16, P, BIG, P, BIG, P, BIG, P, BIG, *s, 2, P, BIG, F16, P, BIG, P, None])
                  for s in ((big, 8, 8), (8, big, 8), (8, 8, big), (8, 2 ** 30, 8))]
        calls += [(L.cr_group_norm, [F16, P, BIG, *s[:2], 1, P, s[2], None, None, 1e-5, 0, P, BIG, None, None, 0, None])
                  for s in ((big, 8, 8), (8, big, 8), (8, 8, big))]
        calls += [(L.cr_group_norm_backward, [F16, P, BIG, *s[:2], 1, P, s[2], None, None, P, BIG, P, P, 8, 0, P, BIG, P, P, None])
                  for s in ((big, 8, 8), (8, big, 8), (8, 8, big))]
        calls += [(L.cr_orthogonalize, [F32, P, BIG, *s, 5, 3.0, -4.0, 2.0, F32, P, BIG, None]) for s in ((big, 8), (8, big))]
        for i, (f, args) in enumerate(calls):
            assert f(*args) == 1, i
            assert "2^31" in L.cr_last_error_detail().decode(), i


def test_nothing_to_do_is_no_error():
    """Zero columns, and gradients that nobody wants, return before any device work."""
    L = cr.load()
    assert L.cr_gated_affine(F16, None, 8, None, 8, 8, 4, 0, None, None, None, 2, F16, None, 0, None, 4, None) == 0
    assert L.cr_group_norm(F16, None, 8, 8, 0, 2, None, 0, None, None, 1e-5, 2, None, 8, None, None, 0, None) == 0
    assert L.cr_gated_affine_backward(F16, P, 8, P, 8, P, 4, P, 8, 8, 4, 2, 2, None, 8, F16, None, 8, None, None) == 0
