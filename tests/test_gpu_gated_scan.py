"""cr_gated_scan, cr_gated_scan_backward and cr_gated_step against the FP64 oracle.

Tolerances.  With e = 2^-19 (the gate's functions to 2^-21 and the rounded operations of a step
and of joining blocks), the state's error obeys E_t = |a| E_{t-1} + e (|a h_{t-1}| + |c x|): the
recurrence itself, run on magnitudes.  The gradients' errors follow from the same recurrence
run backwards.  Outputs are rounded once to their type."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import TYPES, matrix, values, vector, within

pytestmark = pytest.mark.gpu
GATES = ("coeff", "convex", "variance")
E = 2.0 ** -19


def _offsets(rng, T, n):
    cuts = np.sort(rng.integers(0, T + 1, n - 1)) if n > 1 else np.empty(0, int)
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


def _inputs(D, T, n, kind, gate, pad=0, shift=0, seed=0):
    rng = np.random.default_rng(seed + D + T + n)
    g = rng.uniform(-0.99, 0.99, (D, T)) if gate == "coeff" else rng.normal(size=(D, T)) * 2 + 2
    G, X = matrix(g, TYPES[kind], pad, shift), matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift)
    off = _offsets(rng, T, n)
    return rng, G, X, off, matrix(rng.normal(size=(D, n)), torch.float32, pad), torch.from_numpy(off).cuda()


def _state_error(a, c, X, H, off, h0):
    """E_t of the module's docstring, and E before each step."""
    err, before = np.zeros_like(X), np.zeros_like(X)
    for s in range(len(off) - 1):
        e, prev = np.zeros(len(X)), h0[:, s]
        for t in range(off[s], off[s + 1]):
            before[:, t] = e
            e = np.abs(a[:, t]) * e + E * (np.abs(a[:, t] * prev) + np.abs(c[:, t] * X[:, t]))
            prev = H[:, t]
            err[:, t] = e
    return err, before


def _last(err, off, h0):
    return np.stack([err[:, off[s + 1] - 1] if off[s + 1] > off[s] else 0 * h0[:, s] for s in range(len(off) - 1)], axis=1)


def _check(lib, D, T, n, kind, gate, pad=0, shift=0, backward=True):
    rng, G, X, off, h0, doff = _inputs(D, T, n, kind, gate, pad, shift)
    H, hT, saved = lib.gated_scan(G, X, gate, doff, h0, save=True)
    g, x, s0 = values(G), values(X), values(h0)
    Ho, To = trend.gated_scan(g, x, gate, off, s0)
    a, c, da, dc = trend.gate(g, gate)
    err, before = _state_error(a, c, x, Ho, off, s0)
    within(H, Ho, err, TYPES[kind])
    within(hT, To, _last(err, off, s0), torch.float32)
    if not backward:
        return
    dH = matrix(rng.normal(size=(D, T)), TYPES[kind], pad, shift)
    dhT = matrix(rng.normal(size=(D, n)), torch.float32, pad)
    got = lib.gated_scan_backward(G, X, dH, gate, doff, h0, dhT, saved)
    again = lib.gated_scan_backward(G, X, dH, gate, doff, h0, dhT)
    for u, v in zip(got, again):
        assert torch.equal(u, v)   # the states recomputed are the ones saved
    dhv, dtv = values(dH), values(dhT)
    oG, oX, o0 = trend.gated_scan_backward(g, x, dhv, gate, off, s0, dtv)
    eX, eG, e0 = np.zeros_like(x), np.zeros_like(x), np.zeros_like(s0)
    for s in range(n):
        q, eq = dtv[:, s], np.zeros(D)
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            eq = eq + E * (np.abs(q) + np.abs(dhv[:, t]))
            q = q + dhv[:, t]
            prev = Ho[:, t - 1] if t > off[s] else s0[:, s]
            eX[:, t] = np.abs(c[:, t]) * (eq + E * np.abs(q))
            size = np.abs(prev * da[:, t]) + np.abs(x[:, t] * dc[:, t])
            eG[:, t] = (eq + 2 * E * np.abs(q)) * size + (np.abs(q) + eq) * np.abs(da[:, t]) * before[:, t]
            eq = np.abs(a[:, t]) * (eq + E * np.abs(q))
            q = a[:, t] * q
        e0[:, s] = eq
    within(got[0], oG, eG, TYPES[kind])
    within(got[1], oX, eX, TYPES[kind])
    within(got[2], o0, e0, torch.float32)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D,T,n", [(1, 1, 1), (3, 2, 1), (64, 63, 1), (64, 64, 1), (65, 65, 2), (130, 129, 5), (31, 257, 40),
                                   (256, 1000, 3), (2, 3000, 1), (96, 2050, 700), (520, 511, 9)])
def test_scan(lib, kind, gate, D, T, n):
    _check(lib, D, T, n, kind, gate)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (2, 2)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scan_strides(lib, kind, pad, shift):
    for D in (33, 128):
        _check(lib, D, 300, 4, kind, "variance", pad, shift)


@pytest.mark.parametrize("T", [20000, 70001])
def test_scan_long(lib, T):
    """Hundreds of blocks joined along one series, and along a few."""
    _check(lib, 40, T, 1, "bf16", "convex")
    _check(lib, 8, T, 3, "f32", "coeff")


def test_scan_empty_series(lib):
    """Empty series in the middle, in a row, at both ends; no columns at all; no series at all."""
    D = 20
    for off in ([0, 0, 0, 5, 5, 70, 70, 70], [0, 64, 64, 128], [0, 0], [0, 0, 0, 0]):
        T, n = off[-1], len(off) - 1
        rng = np.random.default_rng(n)
        G, X = matrix(rng.normal(size=(D, T)), torch.float16), matrix(rng.normal(size=(D, T)), torch.float16)
        h0, dhT = matrix(rng.normal(size=(D, n)), torch.float32), matrix(rng.normal(size=(D, n)), torch.float32)
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        H, hT, saved = lib.gated_scan(G, X, "convex", o, h0, save=True)
        Ho, To = trend.gated_scan(values(G), values(X), "convex", off, values(h0))
        np.testing.assert_allclose(values(hT), To, rtol=1e-4, atol=1e-5)
        dG, dX, dh0 = lib.gated_scan_backward(G, X, X, "convex", o, h0, dhT, saved)
        _, _, d0 = trend.gated_scan_backward(values(G), values(X), values(X), "convex", off, values(h0), values(dhT))
        np.testing.assert_allclose(values(dh0), d0, rtol=1e-4, atol=1e-4)
        for s in range(n):
            if off[s] == off[s + 1]:
                assert torch.equal(hT[:, s], h0[:, s]) and torch.equal(dh0[:, s], dhT[:, s])
    H, hT = lib.gated_scan(G, X, "convex", torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert H.shape == (D, 0) and hT.shape == (D, 0)


def test_scan_defaults(lib):
    """Without offsets: one series from zero, the same as with them."""
    _, G, X, _, _, _ = _inputs(48, 200, 1, "bf16", "variance")
    H, hT = lib.gated_scan(G, X, "variance")
    o = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    H2, hT2 = lib.gated_scan(G, X, "variance", o, torch.zeros(1, 48, device="cuda").T)
    assert torch.equal(H, H2) and torch.equal(hT, hT2)
    a = lib.gated_scan_backward(G, X, X, "variance")
    b = lib.gated_scan_backward(G, X, X, "variance", o, torch.zeros(1, 48, device="cuda").T, torch.zeros(1, 48, device="cuda").T)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_scan_series_do_not_mix(lib):
    """NaN and infinities in one series leave the other series as they are, bit for bit."""
    D, T = 70, 900
    rng, G, X, _, _, _ = _inputs(D, T, 1, "f32", "coeff")
    off = torch.tensor([0, 100, 333, 333, 700, 900], dtype=torch.int32, device="cuda")
    h0 = matrix(rng.normal(size=(D, 5)), torch.float32)
    dH = matrix(rng.normal(size=(D, T)), torch.float32)
    clean = lib.gated_scan(G, X, "coeff", off, h0, save=True)
    back = lib.gated_scan_backward(G, X, dH, "coeff", off, h0, None, clean[2])
    X2, h2 = X.clone(), h0.clone()
    X2[:, 150] = float("nan")
    X2[:, 250] = float("inf")
    h2[:, 1] = float("inf")
    dirty = lib.gated_scan(G, X2, "coeff", off, h2, save=True)
    back2 = lib.gated_scan_backward(G, X2, dH, "coeff", off, h2, None, dirty[2])
    keep = [t for t in range(T) if not 100 <= t < 333]
    assert torch.equal(dirty[0][:, keep], clean[0][:, keep])
    assert torch.isnan(dirty[0][:, 150:333]).all()
    for u, v in zip(back[:2], back2[:2]):
        assert torch.equal(u[:, keep], v[:, keep])
    assert torch.equal(dirty[1][:, [0, 2, 3, 4]], clean[1][:, [0, 2, 3, 4]])


def test_scan_extreme_gates(lib):
    """Gates at +-inf and far out: a = 1 keeps the state, a = 0 forgets it, nothing overflows."""
    D, T = 16, 300
    for gate in ("convex", "variance"):
        for v, keeps in ((float("inf"), True), (200.0, True), (-200.0, False), (-float("inf"), False)):
            G = torch.full((T, D), v, device="cuda").T
            X = torch.randn(T, D, device="cuda").T
            h0 = torch.randn(1, D, device="cuda").T
            H, hT, saved = lib.gated_scan(G, X, gate, None, h0, save=True)
            want = h0.expand(D, T) if keeps else X
            assert torch.allclose(H, want, rtol=1e-6, atol=1e-6), (gate, v)
            dG, dX, dh0 = lib.gated_scan_backward(G, X, torch.ones_like(X), gate, None, h0, None, saved)
            assert torch.isfinite(dG).all() and torch.isfinite(dX).all() and torch.isfinite(dh0).all()


def test_scan_repeatability_and_streams(lib):
    _, G, X, off, h0, doff = _inputs(300, 5000, 6, "bf16", "convex")
    ref = lib.gated_scan(G, X, "convex", doff, h0, save=True)
    back = lib.gated_scan_backward(G, X, X, "convex", doff, h0, None, ref[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for st in (None, None, s, None):
        got = lib.gated_scan(G, X, "convex", doff, h0, save=True, stream=st)
        gb = lib.gated_scan_backward(G, X, X, "convex", doff, h0, None, got[2], stream=st)
        torch.cuda.synchronize()
        for u, v in zip((*ref, *back), (*got, *gb)):
            assert torch.equal(u, v)


def test_scan_gradient_against_differences(lib):
    """FP32, one direction of the gates: f'' h^2 and FP32 noise / h both stay below 1 % at h = 2^-6."""
    rng, G, X, off, h0, doff = _inputs(24, 150, 3, "f32", "variance")
    dH = matrix(rng.normal(size=(24, 150)), torch.float32)
    Dr = matrix(rng.normal(size=(24, 150)), torch.float32)
    h = 2.0 ** -6
    f = lambda g: float((lib.gated_scan(g, X, "variance", doff, h0)[0].double() * dH.double()).sum())   # noqa: E731
    dG, _, _ = lib.gated_scan_backward(G, X, dH, "variance", doff, h0)
    slope = float((dG.double() * Dr.double()).sum())
    assert abs(slope - (f(G + h * Dr) - f(G - h * Dr)) / (2 * h)) <= 0.01 * max(abs(slope), float(dG.norm()))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D,B,pad", [(1, 1, 0), (33, 7, 0), (128, 3, 0), (1000, 65, 1), (4096, 2, 8)])
def test_step(lib, kind, gate, D, B, pad):
    rng, G, X, _, h, _ = _inputs(D, B, B, kind, gate, pad)
    H, hn = lib.gated_step(G, X, h, gate)
    a, c, _, _ = trend.gate(values(G), gate)
    want = a * values(h) + c * values(X)
    err = E * (np.abs(a * values(h)) + np.abs(c * values(X)))
    within(hn, want, err, torch.float32)
    within(H, want, err, TYPES[kind])
    same = h.T.contiguous().T
    H2, h2 = lib.gated_step(G, X, same, gate, out=same)   # in place
    assert h2.data_ptr() == same.data_ptr() and torch.equal(h2, hn) and torch.equal(H2, H)


def test_step_follows_the_scan(lib):
    _, G, X, _, h0, _ = _inputs(50, 40, 1, "f16", "convex")
    H, hT = lib.gated_scan(G, X, "convex", None, h0)
    h = h0
    for t in range(40):
        y, h = lib.gated_step(G[:, t:t + 1], X[:, t:t + 1], h, "convex")
        # both round the same real recurrence: within the two FP32 errors and one output rounding each
        assert torch.allclose(y.float(), H[:, t:t + 1].float(), rtol=2.0 ** -10, atol=1e-4)
    assert torch.allclose(h, hT, rtol=1e-4, atol=1e-4)
    assert lib.gated_step(G[:, :0], X[:, :0], h0[:, :0])[0].shape == (50, 0)


def test_scan_binding_refusals(lib):
    x = torch.zeros(8, 4, device="cuda").half()
    h = torch.zeros(8, 1, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: lib.gated_scan(x, x.float()), lambda: lib.gated_scan(x, x, "tanh"), lambda: lib.gated_scan(x, x, "convex", off.long()),
                 lambda: lib.gated_scan(x, x, "convex", off, h.half()), lambda: lib.gated_scan(x, x, "convex", off, h[:7]),
                 lambda: lib.gated_scan(x[:, :3], x), lambda: lib.gated_scan_backward(x, x, x, "convex", off, h, None, torch.zeros(3, device="cuda")),
                 lambda: lib.gated_step(x, x, h), lambda: lib.gated_scan(x, x, "convex", off[:1])):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
    assert vector is not None
