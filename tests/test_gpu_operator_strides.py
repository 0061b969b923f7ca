"""Matrices whose leading dimension or number of columns does not fit the library's 32-bit sizes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _far(n, gap):
    """An n x 2 FP16 matrix with columns `gap` elements apart, and a packed copy."""
    base = torch.empty(gap + n, dtype=torch.float16, device="cuda")
    base[:4 * n] = torch.randn(4 * n, device="cuda").half()   # what a wrapped stride would read
    far = base.as_strided((n, 2), (1, gap))
    far.copy_(torch.randn(2, n, device="cuda").half().T)
    return far, far.T.contiguous().T


@pytest.mark.parametrize("gap", [2 ** 31 + 64, 2 ** 32 + 64])
def test_columns_far_apart(lib, gap):
    """Strides of 2^31 elements and more are followed, not cut to 32 bits."""
    x, packed = _far(64, gap)
    g, w = torch.rand(64, device="cuda"), torch.randn(8, 64, device="cuda").half().T
    h = torch.randn(2, 64, device="cuda").T
    assert torch.equal(lib.rmsnorm(x, g)[0], lib.rmsnorm(packed, g)[0])
    assert torch.equal(lib.affine(w, x), lib.affine(w, packed))
    assert torch.equal(lib.gated_scan(x, packed)[0], lib.gated_scan(packed, packed)[0])
    assert torch.equal(lib.gated_step(packed, x, h)[0], lib.gated_step(packed, packed, h)[0])
    with pytest.raises(lib.CrError) as e:
        lib.affine(torch.randn(64, 8, device="cuda").half().T, packed[:8], out=x)
    assert e.value.code == 1


def test_more_columns_than_sizes_hold(lib):
    """Refused, where cut to 32 bits they would be a few columns."""
    n = 2 ** 32 + 8
    x = torch.ones(1, 1, device="cuda").half().expand(1, n)   # no memory of its own
    g, w = torch.ones(1, device="cuda"), torch.ones(1, 1, device="cuda").half()
    for call in (lambda: lib.rmsnorm(x, g), lambda: lib.affine(w, x), lambda: lib.gated_scan(x, x),
                 lambda: lib.gated_step(x, x, x.float()[:, :8])):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1
