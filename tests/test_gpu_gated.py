"""cr_gated_affine and cr_gated_affine_backward against the FP64 oracle.

Tolerances.  Z is a sum of K exact products accumulated in FP32: each addition errs by at most 2^-23 of the sum of
magnitudes S (twice the rounding unit, for adders that truncate), so |dz| <= (K + 8) 2^-23 S.  Activations have slopes
below 1.13 and are evaluated to 2^-20 |z|; the product of both halves is rounded to FP32.  Outputs are rounded once
to their type."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import ROUND, TYPES, matrix, values, vector, within

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu")


def _forward(lib, K, N, M, kind, act="silu", bias=True, out=None, pad=(0, 0, 0), shift=0, save=False):
    rng = np.random.default_rng(K * 7 + N * 3 + M)
    dtype = TYPES[kind]
    out = TYPES[out] if out else (torch.bfloat16 if kind == "e4m3" else dtype)
    W = matrix(rng.normal(size=(K, 2 * N)) * (1.0 if kind == "e4m3" else K ** -0.5), dtype, pad[0], shift)
    X = matrix(rng.normal(size=(K, M)), dtype, pad[1], shift)
    ws = np.float32(rng.uniform(0.5, 2.0, 2 * N) * K ** -0.5) if kind == "e4m3" else None
    xs = np.float32(rng.uniform(0.5, 2.0, M)) if kind == "e4m3" else None
    b = np.float32(rng.normal(size=2 * N)) if bias else None
    place = matrix(np.zeros((N, M)), out, pad[2], shift) if pad[2] or shift else None
    got = lib.gated_affine(W, X, None if b is None else vector(b), act, w_scale=None if ws is None else vector(ws),
                           x_scale=None if xs is None else vector(xs), out_dtype=out, save=save, out=place)
    Y, Z = got if save else (got, None)
    assert place is None or Y.data_ptr() == place.data_ptr()
    Wv, Xv = values(W), values(X)
    Yo, Zo = trend.gated_affine(Wv, Xv, b, act, ws, xs)
    S = np.abs(Wv).T @ np.abs(Xv)
    if kind == "e4m3":
        S = S * ws[:, None] * xs[None, :]
    ez = (K + 8) * 2.0 ** -23 * (S + (0 if b is None else np.abs(b)[:, None]))
    eg = 1.13 * ez[:N] + 2.0 ** -20 * np.abs(Zo[:N])
    ey = eg * (np.abs(Zo[N:]) + ez[N:]) + np.abs(trend.activation(Zo[:N], act)) * ez[N:] + 2.0 ** -22 * np.abs(Yo)
    within(Y, Yo, ey, out)
    if save:
        within(Z, Zo, ez, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("K,N,M", [(1, 1, 1), (7, 5, 3), (64, 128, 1), (100, 33, 2), (128, 256, 8), (257, 129, 16), (512, 384, 17),
                                   (1040, 272, 33), (96, 640, 64), (513, 130, 65), (384, 512, 128), (1024, 96, 129), (200, 260, 300),
                                   (2048, 1024, 1), (640, 2048, 5), (4096, 64, 7), (512, 10000, 1)])
def test_gated_sizes(lib, kind, K, N, M):
    _forward(lib, K, N, M, kind)
    _forward(lib, K, N, M, kind, save=True, bias=False)


@pytest.mark.parametrize("kind,out", [("f16", "f32"), ("bf16", "f16"), ("e4m3", "f32"), ("e4m3", "f16"), ("f16", "f16")])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40, 333])
def test_gated_epilogues(lib, kind, out, act, M):
    _forward(lib, 320, 208, M, kind, act, True, out, save=True)
    _forward(lib, 320, 204, M, kind, act, False, out, save=True)
    _forward(lib, 320, 208, M, kind, act, False, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 12, 200])
@pytest.mark.parametrize("pad,shift", [((16, 16, 16), 0), ((1, 3, 5), 0), ((0, 0, 0), 1), ((8, 1, 2), 8)])
def test_gated_strides(lib, kind, M, pad, shift):
    """Padding and the elements around a matrix are NaN: none may enter."""
    _forward(lib, 272, 144, M, kind, "silu", True, None, pad, shift, save=True)
    _forward(lib, 272, 141, M, kind, "gelu", True, None, pad, shift, save=True)


@pytest.mark.parametrize("K,N,M", [(1536, 2048, 1000), (4096, 515, 2051), (72, 4096, 777), (2048, 200, 4500)])
def test_gated_large(lib, K, N, M):
    _forward(lib, K, N, M, "bf16", "gelu", save=True)
    _forward(lib, K, N, M, "e4m3", "silu", out="f32")


def test_gated_padding_untouched(lib):
    rng = np.random.default_rng(1)
    for K, N, M in ((160, 72, 50), (160, 72, 1), (256, 136, 400), (256, 131, 300)):
        W, X = matrix(rng.normal(size=(K, 2 * N)), torch.float16), matrix(rng.normal(size=(K, M)), torch.float16)
        buf = torch.full((M + 1, N + 9), 7.0, dtype=torch.float16, device="cuda")
        got = lib.gated_affine(W, X, None, "relu", out=buf[:M, :N].T)
        assert got.data_ptr() == buf.data_ptr()
        assert torch.equal(buf[:M, :N].T, lib.gated_affine(W, X, None, "relu"))
        assert (buf[:, N:] == 7.0).all() and (buf[M] == 7.0).all()


def test_gated_exact_integers(lib):
    """Small integers: every product and sum is exact, so the result has no error at all."""
    rng = np.random.default_rng(2)
    for kind in ("f16", "bf16", "e4m3"):
        for K, N, M in ((100, 200, 1), (100, 200, 24), (300, 333, 500)):
            a, b = rng.integers(-4, 5, (K, 2 * N)).astype(float), rng.integers(-4, 5, (K, M)).astype(float)
            Y = lib.gated_affine(matrix(a, TYPES[kind]), matrix(b, TYPES[kind]), act="none", out_dtype=torch.float32)
            z = a.T @ b
            want = z[:N] * z[N:]
            assert np.abs(want).max() < 2 ** 24
            np.testing.assert_array_equal(values(Y), want)


def test_gated_nonfinite(lib):
    """A NaN column of X is NaN in its column only, an infinite gate column of W in its row only."""
    rng = np.random.default_rng(3)
    for M in (1, 3, 200):
        a, b = rng.uniform(0.1, 1, (96, 80)), rng.uniform(0.1, 1, (96, M))
        b[5, 0] = np.nan if M > 1 else 1.0
        a[7, 4] = np.inf
        Y = values(lib.gated_affine(matrix(a, torch.float16), matrix(b, torch.float16), act="silu", out_dtype=torch.float32))
        if M > 1:
            assert np.isnan(Y[:, 0]).all()
            Y = Y[:, 1:]
        assert np.isposinf(Y[4]).all() and np.isfinite(np.delete(Y, 4, axis=0)).all()


def test_gated_halves_of_two_matrices_and_streams(lib):
    """Both projections side by side are one matrix; another stream and repeated calls give the same bits."""
    rng = np.random.default_rng(5)
    wg, wu = rng.normal(size=(200, 700)), rng.normal(size=(200, 700))
    X = matrix(rng.normal(size=(200, 19)), torch.bfloat16)
    W = torch.cat([matrix(wg, torch.bfloat16).T, matrix(wu, torch.bfloat16).T]).T
    ref = lib.gated_affine(W, X, act="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = lib.gated_affine(W, X, act="gelu", stream=s)
    s.synchronize()
    assert torch.equal(ref, other)
    for _ in range(5):
        assert torch.equal(ref, lib.gated_affine(W, X, act="gelu"))
    assert lib.gated_affine(W, X[:, :0]).shape == (700, 0)


def _backward(lib, K, N, M, kind, act, dw=None, pad=0, shift=0):
    rng = np.random.default_rng(K + N + M)
    dtype = TYPES[kind]
    W = matrix(rng.normal(size=(K, 2 * N)) * K ** -0.5, dtype, pad, shift)
    X, dY = matrix(rng.normal(size=(K, M)), dtype, pad, shift), matrix(rng.normal(size=(N, M)), dtype, pad, shift)
    Z = matrix(rng.normal(size=(2 * N, M)), dtype, pad, shift)
    dX, dW, db = lib.gated_affine_backward(W, X, dY, Z, act, dw_dtype=TYPES[dw] if dw else None)
    Wv, Xv, Dv, Zv = values(W), values(X), values(dY), values(Z)
    oX, oW, ob = trend.gated_affine_backward(Wv, Xv, Dv, Zv, act)
    g, h = Zv[:N], Zv[N:]
    G = np.abs(np.concatenate([Dv * h * trend.activation_slope(g, act), Dv * trend.activation(g, act)]))
    u, tiny = ROUND[dtype]
    # slopes are at most 1.13 and err by 2^-19, activations by 2^-20 |z|; G is then rounded to the operands' type (not for db)
    eg = np.concatenate([2.0 ** -19 * np.abs(Dv * h), 2.0 ** -20 * np.abs(Dv * g)]) + 2.0 ** -22 * G
    er = eg + u * (G + eg) + tiny
    within(dX, oX, np.abs(Wv) @ er + (2 * N + 8) * 2.0 ** -23 * (np.abs(Wv) @ (G + er)), dtype)
    within(dW, oW, np.abs(Xv) @ er.T + (M + 8) * 2.0 ** -23 * (np.abs(Xv) @ (G + er).T), TYPES[dw] if dw else dtype)
    within(db, ob, eg.sum(axis=1) + (M + 8) * 2.0 ** -24 * G.sum(axis=1), torch.float32)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("K,N,M", [(1, 1, 1), (33, 20, 7), (128, 64, 40), (256, 200, 300), (300, 129, 513), (1024, 48, 70)])
def test_gated_backward(lib, kind, act, K, N, M):
    _backward(lib, K, N, M, kind, act)
    _backward(lib, K, N, M, kind, act, "f32")


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (3, 8)])
def test_gated_backward_strides(lib, pad, shift):
    _backward(lib, 136, 72, 90, "bf16", "silu", "f32", pad, shift)
    _backward(lib, 520, 264, 600, "f16", "gelu", None, pad, shift)


def test_gated_backward_large_parts_and_empty(lib):
    _backward(lib, 1024, 1500, 2100, "bf16", "silu")
    rng = np.random.default_rng(9)
    K, N, M = 256, 160, 333
    W, X = matrix(rng.normal(size=(K, 2 * N)) * 0.1, torch.float16), matrix(rng.normal(size=(K, M)), torch.float16)
    Z, dY = matrix(rng.normal(size=(2 * N, M)), torch.float16), matrix(rng.normal(size=(N, M)), torch.float16)
    whole = lib.gated_affine_backward(W, X, dY, Z, "gelu")
    for part in range(3):
        need = tuple(q == part for q in range(3))
        got = lib.gated_affine_backward(W, X, dY, Z, "gelu", need)
        for q in range(3):
            assert got[q] is None if q != part else torch.equal(got[q], whole[q])
    assert lib.gated_affine_backward(W, X, dY, Z, "gelu", (False, False, False)) == (None, None, None)
    for a, b in zip(lib.gated_affine_backward(W, X, dY, Z, "gelu"), whole):
        assert torch.equal(a, b)
    dX, dW, db = lib.gated_affine_backward(W, X[:, :0], dY[:, :0], Z[:, :0], "gelu", dw_dtype=torch.float32)
    assert dX.shape == (K, 0) and not dW.any() and not db.any()


def test_gated_gradient_against_differences(lib):
    """FP32 outputs, one direction of a 16-bit X: the step is 2^-3 of exact 16-bit values; the slope's third derivative
    term is below 1 % and the sums err by far less (X, D are multiples of 2^-3 below 2^3: X + D / 8 is exact)."""
    rng = np.random.default_rng(10)
    K, N, M = 64, 48, 30
    W = matrix(np.round(rng.normal(size=(K, 2 * N)) * 16) / 256, torch.float16)
    x, d = np.round(rng.normal(size=(K, M)) * 8) / 8, np.round(rng.normal(size=(K, M)) * 8) / 8
    dY = matrix(np.round(rng.normal(size=(N, M)) * 8) / 8, torch.float16)
    h = 2.0 ** -5
    f = lambda v: float((lib.gated_affine(W, matrix(v, torch.float16), act="silu", out_dtype=torch.float32).double()   # noqa: E731
                         * dY.double()).sum())
    _, Z = lib.gated_affine(W, matrix(x, torch.float16), act="silu", save=True)
    dX, _, _ = lib.gated_affine_backward(W, matrix(x, torch.float16), dY, Z, "silu")
    slope = float((values(dX) * d).sum())
    diff = (f(x + h * d) - f(x - h * d)) / (2 * h)
    assert abs(slope - diff) <= 0.01 * max(abs(slope), float(np.linalg.norm(values(dX))))


def test_gated_binding_refusals(lib):
    x, w, b = torch.zeros(8, 4, device="cuda").half(), torch.zeros(8, 6, device="cuda").half(), torch.ones(6, device="cuda")
    z, dy = torch.zeros(6, 4, device="cuda").half(), torch.zeros(3, 4, device="cuda").half()
    for call in (lambda: lib.gated_affine(w[:, :5], x), lambda: lib.gated_affine(w, x, b[:3]), lambda: lib.gated_affine(w, x, b.half()),
                 lambda: lib.gated_affine(w.float(), x), lambda: lib.gated_affine(w, x, act="tanh"), lambda: lib.gated_affine(w[:7], x),
                 lambda: lib.gated_affine(w, x, w_scale=b), lambda: lib.gated_affine(w.cpu(), x), lambda: lib.gated_affine(w, x.float()),
                 lambda: lib.gated_affine(w, x, out_dtype=torch.float8_e4m3fn), lambda: lib.gated_affine(w, x, out=dy),
                 lambda: lib.gated_affine(w, x, out=z), lambda: lib.gated_affine_backward(w, x, dy, z[:5]),
                 lambda: lib.gated_affine_backward(w, x, z, z), lambda: lib.gated_affine_backward(w[:, :5], x, dy, z),
                 lambda: lib.gated_affine_backward(w, x, dy, z, dw_dtype=torch.bfloat16)):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
