"""The group norm and its gradient with NaN and infinities where a thread's features belong to several groups: odd group sizes in
widths that 16-byte accesses apply to, and more columns than small fields have.  What is not of the bad group has the same bits as
without it."""
import pytest
import torch

from trend_util import TYPES

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
SHAPES = [(64, 64), (24, 8), (40, 8), (56, 8), (256, 8)]   # groups of 1, 3, 5, 7 and 32


def _inputs(D, T, kind, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    return rand(T, D).to(TYPES[kind]).T, rand(T, D).to(TYPES[kind]).T, 1 + 0.2 * rand(D), 0.2 * rand(D), off


def _same(got, want, hit):
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu", "none"])
@pytest.mark.parametrize("D,groups", SHAPES)
@pytest.mark.parametrize("T", [40, 9000])
def test_values_of_x(lib, kind, act, D, groups, T):
    X, dY, gamma, beta, off = _inputs(D, T, kind)
    group = D // groups
    want = lib.group_norm(X, groups, gamma, beta, act, off, save=True)
    back = lib.group_norm_backward(X, groups, gamma, beta, dY, want[1], want[2], act, off)
    for k, value in ((0, NAN), (3, INF), (groups - 1, -INF), (4, NAN)):
        bad = X.clone()
        bad[k * group + group // 2, T // 3 + 7] = value
        got = lib.group_norm(bad, groups, gamma, beta, act, off, save=True)
        rows = slice(k * group, (k + 1) * group)
        hit = torch.zeros(D, T, dtype=torch.bool, device="cuda")
        hit[rows, T // 3:] = True
        _same(got[0], want[0], hit)
        stats = torch.zeros(groups, 3, dtype=torch.bool, device="cuda")
        stats[k, 2] = True
        assert not got[1][stats].isfinite().any() and torch.equal(got[1][~stats], want[1][~stats])   # an infinity's mean is infinite
        _same(got[2], want[2], stats)
        dX, dgamma, dbeta = lib.group_norm_backward(bad, groups, gamma, beta, dY, got[1], got[2], act, off)
        _same(dX, back[0], hit)
        feature = torch.zeros(D, dtype=torch.bool, device="cuda")
        feature[rows] = True
        _same(dgamma, back[1], feature)
        if act in ("silu", "gelu"):   # the others' slopes do not need the value
            _same(dbeta, back[2], feature)
        else:
            assert torch.equal(dbeta[~feature], back[2][~feature])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("D,groups", SHAPES)
@pytest.mark.parametrize("T", [40, 9000])
def test_one_feature_alone(lib, kind, act, D, groups, T):
    """A NaN in beta is its feature's; one in dY is its group's dX and its feature's dgamma and dbeta."""
    X, dY, gamma, beta, off = _inputs(D, T, kind, 1)
    group, i = D // groups, 5
    want, mean, rstd = lib.group_norm(X, groups, gamma, beta, act, off, save=True)
    hit = torch.zeros(D, T, dtype=torch.bool, device="cuda")
    hit[i] = True
    bad = beta.clone()
    bad[i] = NAN
    got = lib.group_norm(X, groups, gamma, bad, act, off)
    assert got[hit].isnan().all()
    # a small field's thread takes two features of a group through one reciprocal: 2^-22 of it, and FP32's or the output's rounding
    u = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}[kind]
    torch.testing.assert_close(got[~hit], want[~hit], rtol=2.0 ** -20 + 2 * u if T == 40 else 0.0, atol=2.0 ** -30 if T == 40 else 0.0)
    back = lib.group_norm_backward(X, groups, gamma, beta, dY, mean, rstd, act, off)
    d = dY.clone()
    d[i, 1] = NAN
    dX, dgamma, dbeta = lib.group_norm_backward(X, groups, gamma, beta, d, mean, rstd, act, off)
    hit[:] = False
    hit[i // group * group:(i // group + 1) * group, :T // 3] = True
    _same(dX, back[0], hit)
    feature = torch.arange(D, device="cuda") == i
    _same(dgamma, back[1], feature)
    _same(dbeta, back[2], feature)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("D,groups", SHAPES)
def test_a_group_of_zeros_without_eps(lib, act, D, groups):
    """0 times infinity: NaN in the group, and nowhere else."""
    T, group = 9000, D // groups
    X, dY, gamma, beta, off = _inputs(D, T, "f32", 2)
    want, mean, rstd = lib.group_norm(X, groups, gamma, beta, act, off, eps=0.0, save=True)
    back = lib.group_norm_backward(X, groups, gamma, beta, dY, mean, rstd, act, off)[0]
    rows = slice(2 * group, 3 * group)
    bad = X.clone()
    bad[rows, :T // 3] = 0.0
    hit = torch.zeros(D, T, dtype=torch.bool, device="cuda")
    hit[rows, :T // 3] = True
    got, mean, rstd = lib.group_norm(bad, groups, gamma, beta, act, off, eps=0.0, save=True)
    _same(got, want, hit)
    assert bool((mean[2, 0] == 0) & (rstd[2, 0] == INF))
    _same(lib.group_norm_backward(bad, groups, gamma, beta, dY, mean, rstd, act, off)[0], back, hit)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("D,groups", SHAPES)
@pytest.mark.parametrize("T", [40, 9000])
def test_an_infinite_scale_is_each_elements_own(lib, act, D, groups, T):
    """gamma = beta = infinity: infinite above the mean, and NaN (infinity less infinity) below it."""
    X, _, gamma, beta, off = _inputs(D, T, "f32", 3)
    i = 2
    want, mean, _ = lib.group_norm(X, groups, gamma, beta, act, off, save=True)
    gamma[i] = beta[i] = INF
    got = lib.group_norm(X, groups, gamma, beta, act, off)
    dev = X[i] - torch.cat([mean[i // (D // groups), 0].expand(T // 3), mean[i // (D // groups), 2].expand(T - T // 3)])
    assert bool((got[i][dev > 1e-4] == INF).all()) and got[i][dev < -1e-4].isnan().all()
    rest = torch.arange(D, device="cuda") != i
    torch.testing.assert_close(got[rest], want[rest], rtol=2.0 ** -20 if T == 40 else 0.0, atol=2.0 ** -30 if T == 40 else 0.0)
