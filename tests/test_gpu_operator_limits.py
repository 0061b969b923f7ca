"""Activations of the affine product and their slopes at infinities and far out, in every output type."""
import numpy as np
import pytest
import torch

from trend_util import values

pytestmark = pytest.mark.gpu
FAR = [-float("inf"), -60000.0, -200.0, 200.0, 60000.0, float("inf")]


@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_limits(lib, out, M, act):
    """0 below, z above, exactly but for the output's one rounding."""
    z = torch.tensor(FAR, device="cuda").half()
    w = torch.zeros(len(FAR), 16, device="cuda").half()
    w[:, 0] = z
    x = torch.zeros(M, 16, device="cuda").half()
    x[:, 0] = 1.0
    w[torch.isinf(z)] = z[torch.isinf(z)][:, None]   # infinity times 0 is NaN: infinite rows throughout
    x[:, 1:] = 2.0 ** -10
    got = values(lib.affine(w.T, x.T, act=act, out_dtype=out))
    want = values(torch.where(z > 0, z.float(), 0.0).to(out))
    np.testing.assert_array_equal(got, np.repeat(want[:, None], M, axis=1))


@pytest.mark.parametrize("kind", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes(lib, kind, act):
    """0 below and 1 above, exactly: the bias's gradient is the sum of dY over the columns above."""
    n = len(FAR)
    Z = torch.tensor(FAR, device="cuda").to(kind).repeat(40, 1).T
    dY = torch.full((40, n), 2.0, device="cuda").to(kind).T
    w = torch.ones(n, 16, device="cuda").to(kind).T
    x = torch.ones(40, 16, device="cuda").to(kind).T
    _, _, db = lib.affine_backward(w, x, dY, Z, act)
    np.testing.assert_array_equal(values(db), [0, 0, 0, 80, 80, 80])
