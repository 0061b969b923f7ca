"""The trend-network operators together: the recurrent-trend example fits, kriges and answers."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_trend.py")
    spec = importlib.util.spec_from_file_location("recurrent_trend", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_recurrent_trend_fits_kriges_and_answers(lib):
    r = _example().main()
    # gradient descent on a smooth objective: the error falls, and below half of where it began
    assert r["losses"][-1] < 0.5 * r["losses"][0]
    # the learned column carries the signal to sites that taught nothing
    assert r["rmse_trend"] < r["rmse_mean"] and r["rmse_kriged"] < r["rmse_mean"]
    # universal kriging is unbiased for the design that it was given: Xo^T W = Xp^T
    n_p, X = r["n_pred"], r["design"]
    np.testing.assert_allclose(X[n_p:].T @ r["weights"], X[:n_p].T, atol=1e-7)
    # e4m3 operands err by 2^-4 at most each, independently along k: a few per cent of the answers
    gap = np.sqrt(np.mean((r["next"] - r["next8"]) ** 2) / np.mean(r["next"] ** 2))
    assert 0 < gap < 0.1
    assert np.isfinite(r["state8"]).all()


def test_step_continues_the_scan(lib):
    """A step from the states of a scan over t columns is the scan over t + 1 columns."""
    import torch
    ex = _example()
    net = ex.RecurrentTrend(8, 64, 3)
    rng = np.random.default_rng(4)
    sites, steps = 20, 7
    x = rng.normal(size=(sites, steps + 1, 8))
    off = lambda t: torch.arange(0, sites * t + 1, t, dtype=torch.int32, device="cuda")        # noqa: E731
    last = lambda t: torch.arange(t - 1, sites * t, t, device="cuda")                          # noqa: E731
    cols = lambda t: ex.columns(x[:, :t].reshape(sites * t, 8).T)                              # noqa: E731
    _, state, _ = net.forward(cols(steps), off(steps), last(steps))
    m, after, _ = net.forward(cols(steps + 1), off(steps + 1), last(steps + 1))
    m1, after1 = net.step(ex.columns(x[:, steps].T), state)
    # the same formulas; BF16 rounds the recurrence's output once in each, 2^-8 of values of order one
    assert torch.allclose(after, after1, rtol=1e-4, atol=1e-4)
    assert torch.allclose(m, m1, rtol=0.05, atol=0.05)
