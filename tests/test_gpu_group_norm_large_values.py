"""The group norm of large finite values: means stay finite, and where the sum of squared deviations passes FP32 the
normalised value is 0, so that y is act(beta) and no gradient reaches X."""
import pytest
import torch

from trend_util import TYPES, values

pytestmark = pytest.mark.gpu


def _offsets(*cuts):
    return torch.tensor(cuts, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 9000, 30011])
@pytest.mark.parametrize("D,groups", [(64, 2), (64, 64), (40, 8), (1000, 1)])
@pytest.mark.parametrize("value", [1e35, 2.0 ** 124])
def test_deviations_beyond_the_squares(lib, kind, T, D, groups, value):
    """Half of each field 0 and half `value`; or of random signs."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    beta = torch.randn(D, generator=gen, device="cuda").to(TYPES[kind]).float()
    gamma = torch.rand(D, generator=gen, device="cuda")
    half = torch.zeros(T, D, device="cuda")
    half[T // 2:] = value
    signs = torch.where(torch.rand(T, D, generator=gen, device="cuda") < 0.5, -value, value)
    dY = torch.randn(T, D, generator=gen, device="cuda").to(TYPES[kind]).T
    for x in (half, signs):
        X = x.to(TYPES[kind]).T
        Y, mean, rstd = lib.group_norm(X, groups, gamma, beta, "none", save=True)
        want = X.double().view(groups, -1, T).mean(dim=(1, 2))
        # sums of n terms of up to `value`: n 2^-24 of it each, tree-like below 2^10 in a row
        assert float((mean[:, 0].double() - want).abs().max()) <= 2.0 ** -13 * value
        assert not rstd.any()
        assert torch.equal(Y, beta[:, None].expand(D, T).to(TYPES[kind]))
        dX, dgamma, dbeta = lib.group_norm_backward(X, groups, gamma, beta, dY, mean, rstd)
        assert not dX.any() and not dgamma.any() and torch.isfinite(dbeta).all()


@pytest.mark.parametrize("T", [40, 9000])
def test_one_far_field_leaves_the_others(lib, T):
    X = torch.randn(2 * T, 48, device="cuda").T.clone()
    off = _offsets(0, T, 2 * T)
    want = lib.group_norm(X, 6, offsets=off)
    X[:, :T // 2] = 3e36
    got = lib.group_norm(X, 6, offsets=off)
    assert torch.equal(got[:, T:], want[:, T:]) and not got[:, :T].any()


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 40])
def test_ordinary_values_of_another_scale(lib, scale):
    """Scaling by a power of two changes no digit."""
    X = torch.randn(9000, 96, device="cuda").T
    Y, mean, rstd = lib.group_norm(X, 6, eps=0.0, save=True)
    y, m, r = lib.group_norm(X * scale, 6, eps=0.0, save=True)
    assert torch.equal(m, mean * scale)
    assert float(((r * scale - rstd) / rstd).abs().max()) <= 2.0 ** -22 and float((y - Y).abs().max()) <= 2.0 ** -20
    assert values(Y).std() > 0.9
