"""cr_affine and cr_affine_backward against the FP64 oracle.

Tolerances.  Z is a sum of K exact products accumulated in FP32: each addition errs by at most
2^-23 of the sum of magnitudes S (twice the rounding unit, for adders that truncate), so
|dz| <= (K + 8) 2^-23 S.  Activations have slopes below 1.13 and are evaluated to 2^-20 |z|.
Outputs are rounded once to their type."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import ROUND, TYPES, matrix, values, vector, within

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu")


def _forward(lib, K, N, M, kind, act, bias, residual, out=None, pad=(0, 0, 0), shift=0, save=False, seed=0):
    rng = np.random.default_rng(seed + K * 7 + N * 3 + M)
    dtype = TYPES[kind]
    out = TYPES[out] if out else (torch.bfloat16 if kind == "e4m3" else dtype)
    W = matrix(rng.normal(size=(K, N)) * (1.0 if kind == "e4m3" else K ** -0.5), dtype, pad[0], shift)
    X = matrix(rng.normal(size=(K, M)), dtype, pad[1], shift)
    ws = np.float32(rng.uniform(0.5, 2.0, N) * K ** -0.5) if kind == "e4m3" else None
    xs = np.float32(rng.uniform(0.5, 2.0, M)) if kind == "e4m3" else None
    b = np.float32(rng.normal(size=N)) if bias else None
    R = matrix(rng.normal(size=(N, M)), out, pad[2], shift) if residual else None
    got = lib.affine(W, X, None if b is None else vector(b), act, R, w_scale=None if ws is None else vector(ws),
                     x_scale=None if xs is None else vector(xs), out_dtype=out, save=save)
    Y, Z = got if save else (got, None)
    Wv, Xv = values(W), values(X)
    Yo, Zo = trend.affine(Wv, Xv, b, act, values(R) if residual else None, ws, xs)
    S = np.abs(Wv).T @ np.abs(Xv)
    if kind == "e4m3":
        S = S * ws[:, None] * xs[None, :]
    ez = (K + 8) * 2.0 ** -23 * (S + (0 if b is None else np.abs(b)[:, None]))
    ey = 1.13 * ez + 2.0 ** -20 * np.abs(Zo) + 2.0 ** -22 * np.abs(Yo)
    within(Y, Yo, ey, out)
    if save:
        within(Z, Zo, ez, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("K,N,M", [(1, 1, 1), (7, 5, 3), (64, 128, 1), (100, 33, 2), (128, 256, 8), (257, 129, 16),
                                   (512, 384, 17), (1040, 272, 33), (96, 640, 64), (513, 130, 65), (384, 512, 128),
                                   (1024, 96, 129), (200, 260, 300), (2048, 1024, 1), (640, 2048, 5), (4096, 64, 7)])
def test_affine_sizes(lib, kind, K, N, M):
    _forward(lib, K, N, M, kind, "none", True, False)


@pytest.mark.parametrize("kind,out", [("f16", "f32"), ("bf16", "f16"), ("e4m3", "f32"), ("e4m3", "f16"), ("f16", "f16")])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 40, 333])
def test_affine_epilogues(lib, kind, out, act, M):
    _forward(lib, 320, 208, M, kind, act, True, True, out, save=True)
    _forward(lib, 320, 208, M, kind, act, False, False, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 12, 200])
@pytest.mark.parametrize("pad,shift", [((16, 16, 16), 0), ((1, 3, 5), 0), ((0, 0, 0), 1), ((8, 1, 2), 8)])
def test_affine_strides(lib, kind, M, pad, shift):
    """Padding and the elements around a matrix are NaN: none may enter, and none is written."""
    _forward(lib, 272, 144, M, kind, "silu", True, True, None, pad, shift, save=True)


@pytest.mark.parametrize("K,N,M", [(1536, 4096, 1000), (4096, 1030, 2051), (72, 8192, 777), (2048, 300, 4500)])
def test_affine_large(lib, K, N, M):
    _forward(lib, K, N, M, "bf16", "gelu", True, True)
    _forward(lib, K, N, M, "e4m3", "none", True, False)


def test_affine_residual_in_place_and_padding_untouched(lib):
    rng = np.random.default_rng(1)
    K, N, M = 160, 72, 50
    W, X = matrix(rng.normal(size=(K, N)), torch.float16), matrix(rng.normal(size=(K, M)), torch.float16)
    buf = torch.full((M, N + 9), 7.0, dtype=torch.float16, device="cuda")
    R = torch.randn(M, N, device="cuda").half()
    buf[:, :N] = R
    view = buf[:, :N].T
    got = lib.affine(W, X, None, "relu", view, out=view)
    assert got.data_ptr() == view.data_ptr()
    assert torch.equal(buf[:, :N].T, lib.affine(W, X, None, "relu", R.T))
    assert (buf[:, N:] == 7.0).all()


def test_affine_exact_integers(lib):
    """Small integers: every product and sum is exact, so the result has no error at all."""
    rng = np.random.default_rng(2)
    for kind in ("f16", "bf16", "e4m3"):
        for K, N, M in ((300, 200, 1), (300, 200, 24), (1000, 333, 500)):
            a, b = rng.integers(-4, 5, (K, N)).astype(float), rng.integers(-4, 5, (K, M)).astype(float)
            Y = lib.affine(matrix(a, TYPES[kind]), matrix(b, TYPES[kind]), out_dtype=torch.float32)
            np.testing.assert_array_equal(values(Y), a.T @ b)


def test_affine_nonfinite(lib):
    """A NaN column of X is NaN in its column only, an infinite row of W in its row only."""
    rng = np.random.default_rng(3)
    for M in (3, 200):
        a, b = rng.uniform(0.1, 1, (96, 40)), rng.uniform(0.1, 1, (96, M))
        b[5, 1] = np.nan
        a[7, 4] = np.inf
        Y = values(lib.affine(matrix(a, torch.float16), matrix(b, torch.float16), act="silu"))
        assert np.isnan(Y[:, 1]).all()
        rest = np.delete(Y, 1, axis=1)
        assert np.isposinf(rest[4]).all() and np.isfinite(np.delete(rest, 4, axis=0)).all()
    # the activations' limits at -inf
    w = torch.full((16, 16), -float("inf"), device="cuda").half()
    x = torch.ones(16, 3, device="cuda").half()
    for act in ("relu", "silu", "gelu"):
        assert (values(lib.affine(w, x, act=act)) == 0).all(), act


def test_affine_streams_and_repeatability(lib):
    rng = np.random.default_rng(5)
    W, X = matrix(rng.normal(size=(2000, 700)), torch.bfloat16), matrix(rng.normal(size=(2000, 19)), torch.bfloat16)
    ref = lib.affine(W, X, act="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = lib.affine(W, X, act="gelu", stream=s)
    s.synchronize()
    assert torch.equal(ref, other)
    for _ in range(5):
        assert torch.equal(ref, lib.affine(W, X, act="gelu"))
    assert lib.affine(W, X[:, :0]).shape == (700, 0)


def _backward(lib, K, N, M, kind, act, dw=None, pad=0, shift=0):
    rng = np.random.default_rng(K + N + M)
    dtype = TYPES[kind]
    W = matrix(rng.normal(size=(K, N)) * K ** -0.5, dtype, pad, shift)
    X, dY = matrix(rng.normal(size=(K, M)), dtype, pad, shift), matrix(rng.normal(size=(N, M)), dtype, pad, shift)
    Z = matrix(rng.normal(size=(N, M)), dtype, pad, shift)
    dX, dW, db = lib.affine_backward(W, X, dY, Z if act != "none" else None, act, dw_dtype=TYPES[dw] if dw else None)
    Wv, Xv, Dv, Zv = values(W), values(X), values(dY), values(Z)
    oX, oW, ob = trend.affine_backward(Wv, Xv, Dv, Zv, act)
    G = np.abs(Dv * trend.activation_slope(Zv, act))
    u, tiny = ROUND[dtype]
    # slopes are at most 1.13 and err by 2^-19; G is then rounded to the operands' type (not for db)
    eg = 0 * G if act == "none" else 2.0 ** -19 * np.abs(Dv)
    er = eg + (0 if act == "none" else u * (G + eg) + tiny)
    within(dX, oX, np.abs(Wv) @ er + (N + 8) * 2.0 ** -23 * (np.abs(Wv) @ (G + er)), dtype)
    within(dW, oW, np.abs(Xv) @ er.T + (M + 8) * 2.0 ** -23 * (np.abs(Xv) @ (G + er).T), TYPES[dw] if dw else dtype)
    within(db, ob, eg.sum(1) + (M + 8) * 2.0 ** -23 * (G + eg).sum(1), torch.float32)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("K,N,M", [(1, 1, 1), (33, 17, 9), (128, 256, 64), (200, 136, 130), (520, 264, 77), (264, 1032, 515)])
def test_affine_backward(lib, kind, act, K, N, M):
    _backward(lib, K, N, M, kind, act)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 3)])
def test_affine_backward_strides_and_wide_gradient(lib, pad, shift):
    _backward(lib, 144, 208, 100, "bf16", "silu", "f32", pad, shift)
    _backward(lib, 144, 208, 100, "f16", "none", "f32", pad, shift)


def test_affine_backward_large(lib):
    _backward(lib, 1024, 2064, 1537, "bf16", "gelu")


def test_affine_backward_parts(lib):
    """Each gradient alone equals its part of the whole call; no columns give zero sums."""
    rng = np.random.default_rng(9)
    W, X = matrix(rng.normal(size=(64, 48)), torch.float16), matrix(rng.normal(size=(64, 80)), torch.float16)
    dY, Z = matrix(rng.normal(size=(48, 80)), torch.float16), matrix(rng.normal(size=(48, 80)), torch.float16)
    whole = lib.affine_backward(W, X, dY, Z, "gelu")
    for i in range(3):
        part = lib.affine_backward(W, X, dY, Z, "gelu", need=tuple(j == i for j in range(3)))
        assert torch.equal(part[i], whole[i]) and all(part[j] is None for j in range(3) if j != i)
    dX, dW, db = lib.affine_backward(W, X[:, :0], dY[:, :0], Z[:, :0], "gelu")
    assert dX.shape == (64, 0) and not dW.any() and not db.any()


@pytest.mark.parametrize("K,N,M,dw", [(768, 2304, 1100, None), (768, 1100, 2304, None), (2048, 2600, 2600, None),
                                      (600, 4100, 300, "f32"), (2048, 600, 5000, "f32")])
def test_affine_backward_products_share_a_round(lib, K, N, M, dw):
    """Both products of a call (the second starts where the first leaves pairs of SMs free) give what each gives alone."""
    gen = torch.Generator("cuda").manual_seed(K + N + M)
    draw = lambda a, b: torch.randn(b, a, device="cuda", generator=gen).bfloat16().T
    W, X, dY, Z = draw(K, N), draw(K, M), draw(N, M), draw(N, M)
    dtype = TYPES[dw] if dw else None
    for act in ("none", "silu"):
        for _ in range(3):
            dX, dW, db = lib.affine_backward(W, X, dY, Z, act, dw_dtype=dtype)
            aX = lib.affine_backward(W, X, dY, Z, act, need=(True, False, False), dw_dtype=dtype)[0]
            aW = lib.affine_backward(W, X, dY, Z, act, need=(False, True, False), dw_dtype=dtype)[1]
            assert torch.equal(dX, aX) and torch.equal(dW, aW)


def test_affine_gradient_against_differences(lib):
    """The gradient of the library's own forward: FP32 outputs, a power-of-two step h along a random
    direction of W (entries of 8 bits, so W + h D is exact in FP16).  f = sum(dY * Y), f'' is
    O(10^3) here, and FP32 sums err by 1e-6 of O(10^3): both below 2 % of f' at h = 2^-8."""
    rng = np.random.default_rng(11)
    K, N, M, h = 64, 32, 48, 2.0 ** -8
    Wv = np.round(rng.normal(size=(K, N)) * 16) / 128
    D = rng.integers(-1, 2, (K, N)).astype(float)
    X, dYv = matrix(rng.normal(size=(K, M)), torch.float16), None
    dY = matrix(rng.normal(size=(N, M)), torch.float16)
    dYv = values(dY)

    def f(w):
        return float(np.sum(dYv * values(lib.affine(matrix(w, torch.float16), X, act="silu", out_dtype=torch.float32))))

    Z = lib.affine(matrix(Wv, torch.float16), X, out_dtype=torch.float16)
    _, dW, _ = lib.affine_backward(matrix(Wv, torch.float16), X, dY, Z, "silu", dw_dtype=torch.float32)
    slope = float(np.sum(values(dW) * D))
    diff = (f(Wv + h * D) - f(Wv - h * D)) / (2 * h)
    assert abs(slope - diff) <= 0.02 * max(abs(slope), np.linalg.norm(values(dW)))


def test_affine_binding_refusals(lib):
    x = torch.zeros(8, 4, device="cuda").half()
    w = torch.zeros(8, 6, device="cuda").half()
    for call in (lambda: lib.affine(w[:7], x), lambda: lib.affine(w.float(), x), lambda: lib.affine(w, x, act="tanh"),
                 lambda: lib.affine(w, x, torch.zeros(5, device="cuda")), lambda: lib.affine(w, x, None, "none", x),
                 lambda: lib.affine(w, x, w_scale=torch.ones(6, device="cuda")), lambda: lib.affine(w, x[0]),
                 lambda: lib.affine(w.cpu(), x), lambda: lib.affine(w, x, out_dtype=torch.float8_e4m3fn),
                 lambda: lib.affine(w, x, out=torch.zeros(6, 4, device="cuda").half()),
                 lambda: lib.affine_backward(w, x, torch.zeros(6, 4, device="cuda").half(), None, "silu")):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
