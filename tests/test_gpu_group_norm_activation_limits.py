"""Activations of the group norm and their slopes far out.  gamma = 0 makes beta the argument itself."""
import numpy as np
import pytest
import torch

from trend_util import ROUND, TYPES, values

pytestmark = pytest.mark.gpu
INF = float("inf")
FAR = [-INF, -60000.0, -200.0, 200.0, 60000.0, INF, -1e30, 1e30]
NEAR = [-86.0, -80.0, -60.0, -50.0, -43.5, -43.0, -42.5, -30.0, -10.0, -3.0, -1.0, -0.125, -1e-6, -1e-30, 0.0, 1e-30, 1e-6, 0.125, 1.0, 3.0,
        10.0, 30.0, 43.0, 86.0]


def _call(lib, beta, kind, T, act):
    D = len(beta)
    X = torch.randn(T, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(TYPES[kind]).T
    gamma, b = torch.zeros(D, device="cuda"), torch.tensor(beta, device="cuda")
    Y, mean, rstd = lib.group_norm(X, 2, gamma, b, act, save=True)
    dY = torch.full((T, D), 2.0, device="cuda").to(TYPES[kind]).T
    dX, _, dbeta = lib.group_norm_backward(X, 2, gamma, b, dY, mean, rstd, act)
    return Y, dX, dbeta


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("T", [40, 9000])
def test_limits(lib, kind, act, T):
    """0 below, z above, slopes 0 and 1, exactly but for the output's one rounding."""
    Y, dX, dbeta = _call(lib, FAR, kind, T, act)
    z = torch.tensor(FAR, device="cuda")
    want = torch.where(z > 0, z, 0.0).to(TYPES[kind])
    assert torch.equal(Y, want[:, None].expand(len(FAR), T)) and not dX.any()
    np.testing.assert_array_equal(values(dbeta), [2.0 * T if v > 0 else 0.0 for v in FAR])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [40, 9000])
def test_silu_between(lib, kind, T):
    """Relative to the value, also where it is tiny: the exponential's argument rounds to |z| 2^-24 (times 1 / ln 2 and ln 2) and the 2^x,
    the reciprocal and their products to 2^-22 or less each, six of them.  The slope sigmoid(z) (1 + z (1 - sigmoid(z))) crosses 0 at
    z = -1.28, where its parts cancel: relative to them.  Sums of T equal terms add T 2^-24."""
    Y, _, dbeta = _call(lib, NEAR, kind, T, "silu")
    z = np.float32(NEAR).astype(float)
    s, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    err = (np.abs(z) + 1) * 2.0 ** -23 + 6 * 2.0 ** -22
    u, tiny = ROUND[TYPES[kind]]
    want = z * s
    assert (np.abs(values(Y) - want[:, None]) <= ((err + u) * np.abs(want) + tiny + 2.0 ** -126)[:, None]).all()
    parts = s * (1 + np.abs(z) * rest)
    assert (np.abs(values(dbeta) - 2 * T * s * (1 + z * rest)) <= 2 * T * ((err + T * 2.0 ** -24) * parts + 2.0 ** -126)).all()
