"""cr_group_norm and cr_group_norm_backward against the FP64 oracle.

Tolerances, u = 2^-24.  A group's mean is joined from at most c = 96 + (shares / 32) partial means, one rounding of at most
the largest magnitude m each: |dmean| <= c u m =: em.  Deviations x - mean err by u m + em =: ed, so the variance v errs
by at most 2 ed sqrt(v) + ed^2 + c u v =: ev, and rstd = (v + eps)^-1/2 by rstd^3 ev / 2 + 2^-22 rstd as long as ev is
below half of v + eps.  h = (x - mean) rstd errs by ed rstd + |x - mean| drstd, gamma h + beta by |gamma| of that and 4 u of
its parts, and activations have slopes below 1.13 and err by 2^-20 |z|.  Outputs are rounded once to their type."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import ROUND, TYPES, matrix, values, vector, within

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu")
U = 2.0 ** -24
# D, groups, offsets
CASES = [(1, 1, [0, 1]), (8, 2, [0, 5]), (24, 3, [0, 1, 1, 2, 40]), (32, 32, [0, 7, 100]), (64, 4, [0, 0, 300, 300]), (100, 5, [0, 33, 50]),
         (160, 8, [0, 700, 1900]), (256, 32, [0, 1024]), (264, 33, [0, 129, 130, 131, 400]), (320, 1, [0, 97, 333]), (640, 32, [0, 515]),
         (1000, 8, [0, 20, 61]), (1024, 1024, [0, 50, 90]), (4096, 16, [0, 3, 17]), (12345, 5, [0, 2, 5])]


def _offsets(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _inputs(D, T, kind, pad=0, shift=0, centre=1.0, seed=0):
    rng = np.random.default_rng(seed + D + 3 * T)
    x = rng.normal(size=(D, T)) * rng.uniform(0.5, 2, (D, 1)) + centre * rng.normal(size=(D, 1))
    return rng, matrix(x, TYPES[kind], pad, shift), np.float32(1 + 0.3 * rng.normal(size=D)), np.float32(0.5 * rng.normal(size=D))


def _spread(v, group):   # a value per group, for its features
    return np.repeat(v, group, axis=0)


def _errors(X, groups, off, mean, rstd, eps):
    """(em, er) by group and field, and ed by feature and field."""
    D = X.shape[0]
    m = np.zeros_like(mean)
    for f in range(len(off) - 1):
        if off[f] < off[f + 1]:
            m[:, f] = np.abs(X[:, off[f]:off[f + 1]]).reshape(groups, -1).max(axis=1)
    c = 96 + max(off) * D / 8 / 32 / 32
    em = c * U * m
    ed = U * m + em
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(rstd > 0, 1 / rstd ** 2 - eps, 0).clip(0)
        ev = 2 * ed * np.sqrt(v) + ed ** 2 + c * U * v
        er = np.where(ev <= 0.5 * (v + eps), 1.5 * rstd ** 3 * ev / 2 + 2.0 ** -22 * rstd, np.inf)
    return em, er, ed


def _check(lib, D, groups, off, kind, act="silu", pad=0, shift=0, centre=1.0, eps=1e-3, affine=True, tail=0):
    T = max(off) + tail
    _, X, gamma, beta = _inputs(D, T, kind, pad, shift, centre)
    place = matrix(np.full((D, T), 3.0), TYPES[kind], pad, shift)
    ref = place.clone()
    Y, mean, rstd = lib.group_norm(X, groups, vector(gamma) if affine else None, vector(beta) if affine else None, act, _offsets(off), eps=eps,
                                   save=True, out=place)
    assert Y is place
    g, b = (gamma.astype(float), beta.astype(float)) if affine else (np.ones(D), np.zeros(D))
    x = values(X)
    y, om, orr = trend.group_norm(x, groups, g, b, act, off, eps)
    em, er, ed = _errors(x, groups, off, om, orr, eps)
    assert np.isfinite(er).all()
    within(mean, om, em, torch.float32)
    within(rstd, orr, er, torch.float32)
    group, err, z = D // groups, np.zeros((D, T)), np.zeros((D, T))
    for f in range(len(off) - 1):
        s = slice(off[f], off[f + 1])
        dev, r = x[:, s] - _spread(om[:, f:f + 1], group), _spread(orr[:, f:f + 1], group)
        eh = _spread(ed[:, f:f + 1], group) * (r + _spread(er[:, f:f + 1], group)) + np.abs(dev) * _spread(er[:, f:f + 1], group)
        z[:, s] = g[:, None] * dev * r + b[:, None]
        err[:, s] = 1.13 * (np.abs(g)[:, None] * eh + 4 * U * (np.abs(g[:, None] * dev * r) + np.abs(b)[:, None])) + 2.0 ** -20 * np.abs(z[:, s])
    n = off[-1]
    within(Y[:, :n], y[:, :n], err[:, :n], TYPES[kind])
    assert torch.equal(Y[:, n:], ref[:, n:])
    assert torch.equal(lib.group_norm(X, groups, vector(gamma) if affine else None, vector(beta) if affine else None, act, _offsets(off),
                                      eps=eps)[:, :n], Y[:, :n])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,groups,off", CASES)
def test_group_norm(lib, kind, D, groups, off):
    _check(lib, D, groups, off, kind)


@pytest.mark.parametrize("act", ACTS)
def test_group_norm_activations(lib, act):
    for affine in (False, True):
        _check(lib, 192, 12, [0, 30, 200], "f16", act, affine=affine)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (16, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_group_norm_strides(lib, kind, pad, shift):
    for D, groups in ((48, 4), (256, 8), (1000, 10)):
        _check(lib, D, groups, [0, 10, 77], kind, "gelu", pad, shift)


def test_group_norm_columns_of_no_field(lib):
    """A padded batch: columns behind the last field are left as they were, and count for nothing."""
    for kind in ("f32", "bf16"):
        _check(lib, 64, 8, [0, 20, 45], kind, tail=19)
        _check(lib, 50, 5, [0, 20, 45], kind, tail=300)
        _check(lib, 64, 8, [0, 0], kind, tail=5)


def test_group_norm_long_and_many(lib):
    rng = np.random.default_rng(2)
    cuts = [0] + sorted(int(c) for c in rng.integers(0, 9001, 300)) + [9001]
    _check(lib, 64, 8, cuts, "bf16")
    _check(lib, 40, 1, [0, 30011], "f16")
    _check(lib, 512, 32, [0, 2000, 9001], "f32", "none")
    _check(lib, 16, 2, list(range(0, 1200)), "bf16")   # fields of one site


def test_group_norm_large_common_value(lib):
    """Deviations 1000 times smaller than the mean keep their digits."""
    _check(lib, 128, 4, [0, 400, 1000], "f32", "none", centre=1000.0, eps=1e-6)


def test_group_norm_constant_and_one_far_value(lib):
    x = np.full((16, 400), 5.0)
    x[8:, :200] = 0.0
    x[8, 0] = 1e4   # the first site far from the rest, which is zero
    X = matrix(x, torch.float32)
    Y, mean, rstd = lib.group_norm(X, 2, offsets=_offsets([0, 200, 400]), eps=1e-3, save=True)
    y, m, r = trend.group_norm(x, 2, np.ones(16), np.zeros(16), "none", [0, 200, 400], 1e-3)
    assert (values(Y)[:, 200:] == 0).all() and (values(Y)[:8] == 0).all()
    np.testing.assert_allclose(values(mean), m, rtol=1e-5)
    np.testing.assert_allclose(values(rstd), r, rtol=1e-5)
    np.testing.assert_allclose(values(Y)[8:, :200], y[8:, :200], rtol=2e-5)


def test_group_norm_nonfinite_stay_in_their_group(lib):
    for T in (40, 3000):
        _, X, gamma, beta = _inputs(64, T, "f32")
        off = _offsets([0, T // 3, T])
        want = lib.group_norm(X, 8, vector(gamma), vector(beta), "silu", off)
        bad = X.clone()
        bad[9, 2], bad[20, T - 1] = float("nan"), float("inf")
        got = lib.group_norm(bad, 8, vector(gamma), vector(beta), "silu", off)
        hit = torch.zeros(64, T, dtype=torch.bool, device="cuda")
        hit[8:16, :T // 3] = True
        hit[16:24, T // 3:] = True
        assert got[hit].isnan().all() and torch.equal(got[~hit], want[~hit])


def test_group_norm_in_place_streams_and_empty(lib):
    _, X, gamma, beta = _inputs(256, 500, "bf16")
    off, g, b = _offsets([0, 100, 100, 450]), vector(gamma), vector(beta)
    want = lib.group_norm(X, 16, g, b, "gelu", off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = lib.group_norm(X, 16, g, b, "gelu", off, stream=s)
    s.synchronize()
    assert torch.equal(other[:, :450], want[:, :450])
    place = X.clone()
    lib.group_norm(place, 16, g, b, "gelu", off, out=place)
    assert torch.equal(place[:, :450], want[:, :450]) and torch.equal(place[:, 450:], X[:, 450:])
    Y, mean, rstd = lib.group_norm(X[:, :0], 16, g, b, "gelu", _offsets([0, 0, 0]), save=True)
    assert Y.shape == (256, 0) and not mean.any() and not rstd.any() and mean.shape == (16, 2)
    Y, mean, rstd = lib.group_norm(X, 16, g, b, "gelu", _offsets([0]), save=True)
    assert mean.shape == (16, 0)
    whole = lib.group_norm(X, 16, g, b, "gelu")
    assert torch.equal(whole, lib.group_norm(X, 16, g, b, "gelu", _offsets([0, 500])))


def _backward(lib, D, groups, off, kind, act="silu", pad=0, shift=0, eps=1e-3, affine=True, tail=0):
    T = max(off) + tail
    rng, X, gamma, beta = _inputs(D, T, kind, pad, shift)
    dY = matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift)
    x, dy = values(X), values(dY)
    g, b = (gamma.astype(float), beta.astype(float)) if affine else (np.ones(D), np.zeros(D))
    _, mean, rstd = trend.group_norm(x, groups, g, b, act, off, eps)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    place = matrix(np.full((D, T), 3.0), TYPES[kind], pad, shift)
    ref = place.clone()
    gv, bv = (vector(gamma), vector(beta)) if affine else (None, None)
    dX, dg, db = lib.group_norm_backward(X, groups, gv, bv, dY, matrix(mean.astype(float), torch.float32), matrix(rstd.astype(float), torch.float32),
                                         act, _offsets(off), out=place)
    assert dX is place
    oX, og, ob = trend.group_norm_backward(x, groups, g, b, dY=dy, mean=mean.astype(float), rstd=rstd.astype(float), act=act, offsets=off)
    # with the same statistics: h errs by 2 u |h| and u |x| r, slopes by 2^-19 and 0.8 of what their arguments do (|act''| <= 0.8; relu's slope
    # jumps where |z| is within its error, which the inputs here stay clear of), sums by their length times u
    group, err, eg, eb = D // groups, np.zeros((D, T)), np.zeros(D), np.zeros(D)
    clear = True
    for f in range(len(off) - 1):
        s, n = slice(off[f], off[f + 1]), off[f + 1] - off[f]
        if n == 0:
            continue
        r = _spread(rstd[:, f:f + 1].astype(float), group)
        h = (x[:, s] - _spread(mean[:, f:f + 1].astype(float), group)) * r
        eh = 2 * U * np.abs(h) + U * np.abs(x[:, s]) * r
        z = g[:, None] * h + b[:, None]
        ez = np.abs(g)[:, None] * eh + 3 * U * (np.abs(g[:, None] * h) + np.abs(b)[:, None])
        if act == "relu":
            clear = clear and (np.abs(z) > ez).all()
        slope = trend.activation_slope(z, act)
        dz = np.abs(dy[:, s] * slope)
        edz = np.abs(dy[:, s]) * (2.0 ** -19 + 0.8 * ez) * (act not in ("none", "relu")) + 2 * U * dz
        c = (n + 64) * U
        eb += edz.sum(axis=1) + c * dz.sum(axis=1)
        eg += (edz * np.abs(h) + dz * eh).sum(axis=1) + c * (dz * np.abs(h)).sum(axis=1)
        w = np.abs(g)[:, None]
        k = (n + group + 64) * U
        one = lambda q: _spread(q.reshape(groups, -1).mean(axis=1)[:, None], group)   # noqa: E731
        m1, m2 = one(w * dz), one(w * dz * np.abs(h))
        e1, e2 = one(w * edz) + k * m1, one(w * (edz * np.abs(h) + dz * eh)) + k * m2
        err[:, s] = r * (w * edz + e1 + np.abs(h) * e2 + eh * m2 + 6 * U * (w * dz + m1 + np.abs(h) * m2))
    assert clear
    total = (len(off) + T / 32 + 64) * U
    n = off[-1]
    within(dX[:, :n], oX[:, :n], err[:, :n], TYPES[kind])
    assert torch.equal(dX[:, n:], ref[:, n:])
    hs = np.zeros((D, T))
    for f in range(len(off) - 1):
        s = slice(off[f], off[f + 1])
        hs[:, s] = (x[:, s] - _spread(mean[:, f:f + 1].astype(float), group)) * _spread(rstd[:, f:f + 1].astype(float), group)
    bound = 1.13 * np.abs(dy[:, :n])
    within(dg, og, eg + total * (bound * np.abs(hs[:, :n])).sum(axis=1), torch.float32)
    within(db, ob, eb + total * bound.sum(axis=1), torch.float32)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,groups,off", CASES)
def test_group_norm_backward(lib, kind, D, groups, off):
    _backward(lib, D, groups, off, kind)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_group_norm_backward_activations(lib, act):
    for affine in (False, True):
        _backward(lib, 192, 12, [0, 30, 200], "f16", act, affine=affine)


def test_group_norm_backward_relu(lib):
    _backward(lib, 48, 6, [0, 30, 60], "f32", "relu")


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1)])
def test_group_norm_backward_strides(lib, pad, shift):
    for D, groups in ((48, 4), (256, 8), (1000, 10)):
        _backward(lib, D, groups, [0, 10, 77], "bf16", "gelu", pad, shift, tail=9)


def test_group_norm_backward_long_and_many(lib):
    rng = np.random.default_rng(2)
    cuts = [0] + sorted(int(c) for c in rng.integers(0, 5001, 200)) + [5001]
    _backward(lib, 64, 8, cuts, "bf16")
    _backward(lib, 40, 1, [0, 20011], "f16")
    _backward(lib, 512, 32, [0, 2000, 6001], "f32", tail=100)


def test_group_norm_backward_parts_in_place_and_empty(lib):
    rng, X, gamma, beta = _inputs(320, 300, "f16")
    off, g, b = _offsets([0, 120, 300]), vector(gamma), vector(beta)
    dY = matrix(rng.normal(size=(320, 300)), torch.float16)
    _, mean, rstd = lib.group_norm(X, 20, g, b, "silu", off, save=True)
    whole = lib.group_norm_backward(X, 20, g, b, dY, mean, rstd, "silu", off)
    for part in range(3):
        need = tuple(q == part for q in range(3))
        got = lib.group_norm_backward(X, 20, g, b, dY, mean, rstd, "silu", off, need)
        for q in range(3):
            assert got[q] is None if q != part else torch.equal(got[q], whole[q])
    for place in (dY.clone(), X.clone()):
        on_dy = torch.equal(place, dY)
        got = lib.group_norm_backward(X if on_dy else place, 20, g, b, place if on_dy else dY, mean, rstd, "silu", off, out=place)
        assert got[0] is place and all(torch.equal(p, q) for p, q in zip(got, whole))
    wide = torch.zeros(2, 37, device="cuda")
    strided = (wide[:, :20].copy_(mean.T).T, rstd)
    for p, q in zip(lib.group_norm_backward(X, 20, g, b, dY, *strided, "silu", off), whole):
        assert torch.equal(p, q)
    dX, dg, db = lib.group_norm_backward(X[:, :0], 20, g, b, dY[:, :0], mean[:, :1], rstd[:, :1], "silu", _offsets([0, 0]))
    assert dX.shape == (320, 0) and not dg.any() and not db.any()


def test_group_norm_gradient_against_differences(lib):
    """FP32, one direction: f''' h^2 / 6 and FP32 sums of about 1e-6 / h of f, both below 1 % at 2^-7."""
    rng, X, gamma, beta = _inputs(96, 60, "f32")
    dY, D = matrix(rng.normal(size=(96, 60)), torch.float32), matrix(rng.normal(size=(96, 60)), torch.float32)
    g, b, h, off = vector(gamma), vector(beta), 2.0 ** -7, _offsets([0, 25, 60])
    f = lambda x: float((lib.group_norm(x, 8, g, b, "gelu", off).double() * dY.double()).sum())   # noqa: E731
    _, mean, rstd = lib.group_norm(X, 8, g, b, "gelu", off, save=True)
    dX, _, _ = lib.group_norm_backward(X, 8, g, b, dY, mean, rstd, "gelu", off)
    slope = float((dX.double() * D.double()).sum())
    diff = (f(X + h * D) - f(X - h * D)) / (2 * h)
    assert abs(slope - diff) <= 0.01 * max(abs(slope), float(dX.norm()))


def test_group_norm_binding_refusals(lib):
    x, g = torch.zeros(8, 4, device="cuda").half(), torch.ones(8, device="cuda")
    off, m = _offsets([0, 4]), torch.ones(2, 1, device="cuda")
    for call in (lambda: lib.group_norm(x, 3, g, g), lambda: lib.group_norm(x, 0, g, g), lambda: lib.group_norm(x, 2, g[:7], g),
                 lambda: lib.group_norm(x, 2, g.half(), g), lambda: lib.group_norm(x, 2, g, g, "tanh"),
                 lambda: lib.group_norm(x, 2, g, g, offsets=off.long()), lambda: lib.group_norm(x, 2, g, g, offsets=off.cpu()),
                 lambda: lib.group_norm(x.double(), 2, g, g), lambda: lib.group_norm(x, 2, g, g, eps=-1.0),
                 lambda: lib.group_norm(x, 2, g, g, out=x.float()), lambda: lib.group_norm(x, 2, g, g, out=x.T.contiguous().T[:, :3]),
                 lambda: lib.group_norm(x, 2, g.cpu(), g), lambda: lib.group_norm_backward(x, 2, g, g, x.float(), m, m),
                 lambda: lib.group_norm_backward(x, 2, g, g, x, m[:1], m), lambda: lib.group_norm_backward(x, 2, g, g, x, m.half(), m),
                 lambda: lib.group_norm_backward(x, 5, g, g, x, m, m)):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
    assert ROUND
