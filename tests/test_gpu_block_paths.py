"""The operators' other kernels at the alignments and sizes where they change over: the group norm of many columns with any
strides, and the orthogonalised update by few-tile products, by parts of k and by half tiles, into any matrix.  Tolerances
are those of the operators' own tests."""
import numpy as np
import pytest
import torch

from test_gpu_group_norm import _backward as norm_backward
from test_gpu_group_norm import _check as norm
from test_gpu_orthogonalize import _check as update
from test_gpu_orthogonalize import _gradient
from trend_util import TYPES, matrix, values

pytestmark = pytest.mark.gpu
CUBIC = (1.5, -0.5, 0.0)   # a bound that stays small over large matrices


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (4, 4), (1, 0), (0, 1)])
def test_group_norm_of_many_columns(lib, kind, pad, shift):
    norm(lib, 96, 4, [0, 900, 901, 2500], kind, "silu", pad, shift, tail=3)
    norm(lib, 136, 8, [0, 1700], kind, "gelu", pad, shift)
    norm(lib, 333, 3, [0, 40, 800], kind, "relu", pad, shift)
    norm_backward(lib, 136, 8, [0, 700, 1700], kind, "gelu", pad, shift, tail=3)


@pytest.mark.parametrize("D,groups", [(1000, 1), (808, 8), (808, 101), (640, 32), (72, 72), (2056, 257)])
def test_group_norm_groups_across_tiles(lib, D, groups):
    norm(lib, D, groups, [0, 130, 1500], "bf16")
    norm_backward(lib, D, groups, [0, 130, 700], "bf16")


def test_group_norm_many_small_fields(lib):
    """A launch for small fields, and one with fields of one to three sites in every tile."""
    rng = np.random.default_rng(1)
    for fields, D, groups in ((157, 2304, 32), (2000, 24, 3)):
        cuts = np.cumsum(rng.integers(0, 4, fields)).tolist()
        norm(lib, D, groups, [0] + cuts, "f16", tail=2)
    cuts = np.cumsum(rng.integers(0, 4, 3000)).tolist()
    norm(lib, 64, 2, [0] + cuts, "bf16")
    norm_backward(lib, 64, 2, [0] + cuts[:500], "bf16")


@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (1, 0), (0, 1), (3, 8)])
@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16")])
def test_update_of_medium_matrices(lib, kind, out, pad, shift):
    for K, N in ((200, 333), (700, 260), (140, 2200)):
        place = matrix(np.zeros((K, N)), TYPES[out], pad, shift)
        got, _ = update(lib, matrix(_gradient(K, N), TYPES[kind], pad, shift), out, 1, CUBIC, place=place)
        assert got is place


@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("K,N", [(1301, 1400), (1600, 1250)])
def test_update_of_large_matrices_into_any_matrix(lib, K, N, pad, shift):
    for out in ("bf16", "f32"):
        place = matrix(np.zeros((K, N)), TYPES[out], pad, shift)
        got, _ = update(lib, matrix(_gradient(K, N), torch.float32, pad, shift), out, 2, CUBIC, place=place)
        assert got is place


@pytest.mark.parametrize("K,N", [(100, 5000), (4500, 90), (128, 8192), (129, 128), (128, 129), (1, 9000), (9000, 2)])
def test_update_of_long_matrices(lib, K, N):
    """Where a cluster ends, and products of few rows begin."""
    G = matrix(_gradient(K, N), torch.float32)
    update(lib, G, "f32", 1, CUBIC)
    update(lib, G, "bf16", 1, CUBIC)


def test_update_symmetry_and_order_of_columns(lib):
    """The update of a permuted matrix is the permuted update, and that of the transposed one the transposed update, to the rounding of
    the matrices between the products (2^-21 for two FP16 parts, grown by less than 64 over three steps)."""
    for K, N in ((90, 300), (260, 700), (1000, 1100)):
        g = np.float32(_gradient(K, N)).astype(float)
        a = values(lib.orthogonalize(matrix(g, torch.float32), 3))
        b = values(lib.orthogonalize(matrix(g.T.copy(), torch.float32), 3)).T
        order = np.random.default_rng(3).permutation(N)
        c = values(lib.orthogonalize(matrix(g[:, order], torch.float32), 3))
        for other in (b, c[:, np.argsort(order)]):
            assert np.linalg.norm(other - a) <= 64 * 2.0 ** -21 * np.linalg.norm(a) * np.sqrt(3)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_update_of_millions_of_columns(lib, out):
    """r copies of H side by side: A is H's, X is H's over sqrt(r), and so is each copy's update.  Both sides carry the same roundings,
    of other values: twice what the symmetry test allows for FP32, twice the BF16 test's bound below for BF16."""
    H, r = matrix(_gradient(160, 1000), torch.float32), 2200
    want = lib.orthogonalize(H, 1, out_dtype=out).float()
    G = H.T.repeat(r, 1).T
    got = lib.orthogonalize(G, 1, out_dtype=out)
    limit = 2 * 64 * 2.0 ** -21 if out is torch.float32 else 2 * (2.0 ** -8 + 4 * 2.0 ** -11)
    for block in (got[:, :1000], got[:, -1000:], got[:, 1000 * (r // 2):1000 * (r // 2 + 1)]):
        assert float((block.float() * r ** 0.5 - want).norm()) <= limit * float(want.norm())


def test_update_of_entries_of_all_sizes(lib):
    """Entries from 2^-140 to 2^120 in one matrix: the large ones are all that counts, wherever they lie; and a matrix of 2^49, whose
    squares' sum passes FP32's range."""
    for K, N in ((60, 100), (300, 520)):
        g = np.float32(_gradient(K, N)).astype(float)
        for big, small in ((120, -140), (60, -40), (0, -60), (-60, -130)):
            both = g * 2.0 ** big
            both[:, N // 2:] *= 2.0 ** (small - big)
            want = lib.orthogonalize(matrix(np.where(np.arange(N) < N // 2, g, 0.0), torch.float32), 2)
            got = lib.orthogonalize(matrix(both, torch.float32), 2)
            assert np.linalg.norm(values(got)[:, :N // 2] - values(want)[:, :N // 2]) <= 1e-3 * np.linalg.norm(values(want))
            assert np.isfinite(values(got)).all()
    n = 2 ** 14 + 2 ** 12
    x = torch.full((n, n), 2.0 ** 49, device="cuda", dtype=torch.bfloat16).T
    got = lib.orthogonalize(x, 1, (1.0, 0.0, 0.0))   # G / |G|_F
    assert torch.allclose(got.float(), torch.full_like(got, 1.0 / n).float(), rtol=2 ** -8)
