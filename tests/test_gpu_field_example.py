"""examples/field_trend.py: it runs, and its gradients are those of its loss."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "field_trend.py")
    spec = importlib.util.spec_from_file_location("field_trend", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_field_trend_runs(lib):
    r = _example().main(sites=256, observed=192, fields=5, rounds=6)
    assert len(r["losses"]) == 6 and np.isfinite(r["losses"]).all()
    assert r["kriged"].shape == (64,) and np.isfinite(r["kriged"]).all() and np.isfinite(r["design"]).all()


def test_field_trend_gradients(lib):
    """Against a PyTorch FP32 form of the block, differentiated by autograd, at the same BF16 weights: BF16 matrices between the operators
    are each off by 2^-9 of their size on average, and no gradient passes more than ten of them; they do not add up beyond
    their number: 10 * 2^-9 = 0.02, allowed twice."""
    ex = _example()
    rng = np.random.default_rng(2)
    net = ex.FieldTrend(16, 64, 96, 1)
    X = ex.columns(rng.normal(size=(16, 300)))
    off = torch.tensor([0, 90, 90, 220, 300], dtype=torch.int32, device="cuda")
    dm = torch.from_numpy(rng.normal(size=300)).float().cuda()
    m, kept = net.forward(X, off)
    grads = net.gradients(dm, kept)
    p = {n: (net.w[n].float() if n in net.w else t.clone()).detach().requires_grad_() for n, t in net.master.items()}
    A = p["W1"].T @ X.float() + p["b1"][:, None]
    parts = []
    for a, b in ((0, 90), (90, 220), (220, 300)):
        block = A[:, a:b].reshape(ex.GROUPS, -1)
        h = ((block - block.mean(1, keepdim=True)) / torch.sqrt(block.var(1, unbiased=False, keepdim=True) + 1e-5)).reshape(64, b - a)
        z = p["gamma"][:, None] * h + p["beta"][:, None]
        parts.append(z * torch.sigmoid(z))
    Z = p["W23"].T @ torch.cat(parts, 1)
    V = Z[:96] * torch.sigmoid(Z[:96]) * Z[96:]
    out = (p["Wh"].T @ (p["Wd"].T @ V + A))[0] + p["bh"]
    assert float((out.detach() - m).norm()) <= 0.04 * float(out.detach().norm())
    (out * dm).sum().backward()
    for n, g in grads.items():
        want = p[n].grad
        assert float((g - want).norm()) <= 0.04 * float(want.norm()), n
