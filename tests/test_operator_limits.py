"""Sizes of the trend-network operators: each entry refuses, before any device work, sizes so near
2^31 that its kernels' 32-bit indices would pass it (host only)."""
import pytest

import mixed_precision_dense_mat_gb300 as cr

BIG = 2 ** 31 - 1
P = 4096   # never dereferenced: the calls end at their checks
F16, F32, E4M3 = 1, 0, 3


def _calls(big):
    """Each entry with `big` in place of each of its sizes."""
    def affine(K, N, M):
        return cr._lib.cr_affine(F16, P, BIG, P, BIG, K, N, M, None, None, None, 0, F16, None, 0, None, 0, P, BIG, None)

    def affine_backward(K, N, M):
        return cr._lib.cr_affine_backward(F16, P, BIG, P, BIG, P, BIG, P, BIG, K, N, M, 2, P, BIG, F16, P, BIG, P, None)

    def rmsnorm(D, T):
        return cr._lib.cr_rmsnorm(F16, P, BIG, None, 0, P, D, T, 1e-6, None, 0, F16, P, BIG, None, None)

    def rmsnorm_backward(D, T):
        return cr._lib.cr_rmsnorm_backward(F16, P, BIG, P, P, BIG, None, 0, D, T, 1e-6, P, BIG, P, None)

    def scan(D, T, n):
        return cr._lib.cr_gated_scan(F16, 0, P, BIG, P, BIG, D, T, P, n, None, 0, P, BIG, P, BIG, None, None)

    def scan_backward(D, T, n):
        return cr._lib.cr_gated_scan_backward(F16, 0, P, BIG, P, BIG, P, BIG, D, T, P, n, None, 0, None, 0, P, P, BIG, P, BIG, P,
                                              BIG, None)

    def step(D, B):
        return cr._lib.cr_gated_step(F16, 0, P, BIG, P, BIG, P, BIG, D, B, None, 0, P, BIG, None)

    for f, sizes in ((affine, 3), (affine_backward, 3), (rmsnorm, 2), (rmsnorm_backward, 2), (scan, 3), (scan_backward, 3), (step, 2)):
        for i in range(sizes):
            yield f"{f.__name__}, size {i}", f, [big if j == i else 8 for j in range(sizes)]


@pytest.mark.parametrize("big", [BIG, 2 ** 31 - 2 ** 16 + 1])
def test_sizes_near_two_to_the_31_are_refused(big):
    cr.load()
    for name, f, sizes in _calls(big):
        assert f(*sizes) == 1, name
        assert "2^31" in cr._lib.cr_last_error_detail().decode(), name
