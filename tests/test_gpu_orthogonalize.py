"""cr_orthogonalize against the FP64 closed form by singular values.

Tolerance, in the Frobenius norm |.|.  One step p(X) = a X + (b A + c A^2) X maps an error e of X to at most L |e|, L the
largest of |p(s) - p(t)| / |s - t|, (p(s) + p(t)) / (s + t) and p(s) / s over X's singular values (Daleckii and Krein's
formula), and adds its own: with u the rounding of the matrices between the products (2^-11 for one FP16 part; 2^-21
for two, the product of the two second parts included) and w = (1.01 k + 8) 2^-23 for FP32 sums of k products (twice the
rounding unit, for adders that truncate; with two parts the 2 k products with a second part are summed first: their sums stay
below 2^-10 of the whole sum of magnitudes, so that their additions err by 2 k 2^-33 of it),
    A:  dA <= (u + w) |abs(X) abs(X)^T|,
    B = b A + c A A:  dB <= (|b| + 2 |c| max A) dA + (u + w) (|b| |A| + |c| |abs(A) abs(A)|),
    X': max X dB + (u + w) (|a| |X| + |abs(B) abs(X)|),
max being the largest singular value, and an FP16 entry is off by at least 2^-35 (its scaled spacing).  The last step rounds
to the output's type.  The bounds are followed step by step with the exact matrices; second-order terms are allowed for by a
factor of 2, and a bound above 0.3 of the result's norm would say nothing, so the cases are chosen below it."""
import numpy as np
import pytest
import torch

from oracle import trend
from trend_util import ROUND, TYPES, matrix, values

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)


def _bound(G, steps, coeffs, pairs):
    a, b, c = coeffs
    u = 2.0 ** -21 if pairs else 2.0 ** -11
    x = G / np.linalg.norm(G)
    if x.shape[0] > x.shape[1]:
        x = x.T
    n, k = x.shape
    tiny = 2.0 ** -35 * np.sqrt(n * k)
    norm = np.linalg.norm
    e = u * norm(x) + tiny
    for _ in range(steps):
        s = np.linalg.svd(x, compute_uv=False)
        p = s * (a + s * s * (b + c * s * s))
        ds, dp = s[:, None] - s[None, :], p[:, None] - p[None, :]
        slope = np.abs(a + 3 * b * s * s + 5 * c * s ** 4)
        apart = np.abs(ds) > 1e-9 * s[0]
        L = max(slope.max(), np.abs(np.where(apart, dp / np.where(apart, ds, 1), 0)).max(),
                (np.abs(p[:, None] + p[None, :]) / np.maximum(s[:, None] + s[None, :], 1e-300)).max(), np.abs(a + b * s * s + c * s ** 4).max())
        A = x @ x.T
        B = b * A + c * A @ A
        wk, wn = (1.01 * k + 8) * 2.0 ** -23, (1.01 * n + 8) * 2.0 ** -23
        X_, A_, B_ = np.abs(x), np.abs(A), np.abs(B)
        dA = (u + wk) * norm(X_ @ X_.T) + tiny
        dB = (abs(b) + 2 * abs(c) * s[0] ** 2) * dA + (u + wn) * (abs(b) * norm(A) + abs(c) * norm(A_ @ A_)) + tiny
        y = a * x + B @ x
        e = L * e + s[0] * dB + (u + wn) * (abs(a) * norm(x) + norm(B_ @ X_)) + u * norm(y) + tiny
        x = y
    return 2 * e


def _check(lib, G, out, steps=5, coeffs=COEFFS, pad=0, shift=0, place=None):
    got = lib.orthogonalize(G, steps, coeffs, out_dtype=TYPES[out], out=place)
    g = values(G)
    want = trend.orthogonalize(g, steps, coeffs)
    err = _bound(g, steps, coeffs, out != "bf16")
    assert err < 0.3 * np.linalg.norm(want), "the case says nothing"
    u, tiny = ROUND[TYPES[out]]
    limit = err + u * (np.linalg.norm(want) + err) + tiny * np.sqrt(want.size)
    assert np.linalg.norm(values(got) - want) <= limit, (np.linalg.norm(values(got) - want), limit)
    return got, want


def _gradient(K, N, seed=0):
    """Singular values between 0.3 and 1 of a common size."""
    rng = np.random.default_rng(seed + K + 3 * N)
    q, _ = np.linalg.qr(rng.normal(size=(max(K, N), min(K, N))))
    r, _ = np.linalg.qr(rng.normal(size=(min(K, N), min(K, N))))
    g = (q * rng.uniform(0.3, 1, min(K, N))) @ r * 0.02
    return g if K >= N else g.T


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f16")])
@pytest.mark.parametrize("K,N", [(1, 1), (5, 3), (1, 40), (64, 64), (33, 100), (130, 60), (128, 128), (200, 333), (500, 129), (257, 511), (300, 1100),
                                 (1000, 260)])
def test_orthogonalize(lib, kind, out, K, N):
    _check(lib, matrix(_gradient(K, N), TYPES[kind]), out, 3)
    _check(lib, matrix(_gradient(K, N), TYPES[kind]), out, 1)


@pytest.mark.parametrize("K,N", [(40, 64), (128, 128), (300, 200), (640, 1030)])
def test_orthogonalize_five_steps(lib, K, N):
    got, want = _check(lib, matrix(_gradient(K, N), torch.float32), "f32")
    s = np.linalg.svd(values(got), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.25   # the coefficients' range
    # one 16-bit part: the same to the closed form's error of the pairs' result and a few roundings
    b = values(lib.orthogonalize(matrix(_gradient(K, N), torch.float32), out_dtype=torch.bfloat16))
    assert np.linalg.norm(b - want) <= 0.02 * np.linalg.norm(want)


@pytest.mark.parametrize("K,N", [(2100, 2300), (2600, 1800)])
def test_orthogonalize_large(lib, K, N):
    """Symmetric products by half of their tiles.  Classic cubic coefficients keep the bound small."""
    G = matrix(_gradient(K, N), torch.float32)
    _check(lib, G, "f32", 2, (1.5, -0.5, 0.0))
    _check(lib, G, "bf16", 2, (1.5, -0.5, 0.0))
    _check(lib, G, "f32", 2)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (3, 8)])
def test_orthogonalize_strides(lib, pad, shift):
    for K, N in ((136, 72), (70, 131), (64, 300)):
        for kind, out in (("f32", "f32"), ("bf16", "bf16"), ("f16", "f16")):
            place = matrix(np.zeros((K, N)), TYPES[out], pad, shift)
            got, _ = _check(lib, matrix(_gradient(K, N), TYPES[kind], pad, shift), out, 2, place=place)
            assert got is place


def test_orthogonalize_padding_untouched_and_in_place(lib):
    for K, N in ((130, 90), (600, 700)):
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            buf = torch.full((N + 1, K + 5), 7.0, dtype=dtype, device="cuda")
            G = matrix(_gradient(K, N), dtype)
            want = lib.orthogonalize(G)
            lib.orthogonalize(G, out=buf[:N, :K].T)
            assert torch.equal(buf[:N, :K].T, want) and (buf[:, K:] == 7.0).all() and (buf[N] == 7.0).all()
            lib.orthogonalize(G, out=G)
            assert torch.equal(G, want)


def test_orthogonalize_scale_zero_and_nonfinite(lib):
    """Any size of G, from squares that underflow to ones that overflow, gives the same; zeros, NaN and infinity as documented."""
    for K, N in ((60, 100), (300, 280)):
        g = _gradient(K, N)
        want = lib.orthogonalize(matrix(g, torch.float32))
        for e in (-130, -100, -60, 60, 100, 126):
            got = lib.orthogonalize(matrix(g * 2.0 ** e, torch.float32))
            if e > -130:   # exact scaling: the same up to FP32's rounding of the norm
                assert torch.equal(got, lib.orthogonalize(matrix(g, torch.float32) * 2.0 ** e))
            assert np.linalg.norm(values(got) - values(want)) <= 1e-3 * np.linalg.norm(values(want)), e
        zero = torch.zeros(N, K, device="cuda").T
        assert not lib.orthogonalize(zero).any()
        for bad in (float("nan"), float("inf")):
            G = matrix(g, torch.float32)
            G[3, 5] = bad
            for out in (torch.float32, torch.bfloat16):
                assert lib.orthogonalize(G, out_dtype=out).isnan().all()
        assert torch.isfinite(lib.orthogonalize(matrix(g, torch.float32))).all()   # nothing stays behind


def test_orthogonalize_streams_and_repeatability(lib):
    for K, N in ((128, 128), (700, 1300)):
        G = matrix(_gradient(K, N), torch.float32)
        for out in (torch.float32, torch.bfloat16):
            want = lib.orthogonalize(G, out_dtype=out)
            torch.cuda.synchronize()
            s = torch.cuda.Stream()
            other = lib.orthogonalize(G, out_dtype=out, stream=s)
            s.synchronize()
            assert torch.equal(other, want)
            for _ in range(3):
                assert torch.equal(lib.orthogonalize(G, out_dtype=out), want)


def test_orthogonalize_binding_refusals(lib):
    x = torch.ones(8, 4, device="cuda").T
    for call in (lambda: lib.orthogonalize(x.double()), lambda: lib.orthogonalize(x.cpu()), lambda: lib.orthogonalize(x, 0),
                 lambda: lib.orthogonalize(x, 5, (float("nan"), 0, 0)), lambda: lib.orthogonalize(x, 5, (100.0, 0, 0)),
                 lambda: lib.orthogonalize(x[:, :0]), lambda: lib.orthogonalize(x, out=x[:3]), lambda: lib.orthogonalize(x[0]),
                 lambda: lib.orthogonalize(x, out_dtype=torch.float8_e4m3fn), lambda: lib.orthogonalize(x, out=x.T.contiguous())):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
