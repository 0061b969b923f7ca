"""Waits that surely run out with a limit of zero (CR_OPT_WAIT_LIMIT_US): products long enough that a warp waits for longer than one
try.  Each such call is reported by the next one, once, which does nothing; after it the same bits as before."""
import pytest
import torch

from test_gpu_faults import option

pytestmark = pytest.mark.gpu
H, B, F32 = torch.float16, torch.bfloat16, torch.float32


def _m(k, n, dtype, seed):
    return torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").mul_(k ** -0.5).to(dtype).T


def _call(lib, name):
    if name == "gated, few columns":
        w, x = _m(2 ** 20, 64, H, 1), _m(2 ** 20, 16, H, 2)
        return lambda: lib.gated_affine(w, x, save=True)
    if name == "gated, many columns":
        w, x = _m(2 ** 16, 512, H, 3), _m(2 ** 16, 700, H, 4)
        return lambda: lib.gated_affine(w, x, save=True)
    if name == "gated, gradient":
        w, x, d, z = _m(700, 512, H, 5), _m(700, 2 ** 16, H, 6), _m(256, 2 ** 16, H, 7), _m(512, 2 ** 16, H, 8)
        return lambda: lib.gated_affine_backward(w, x, d, z)
    if name == "affine, few columns":
        w, x = _m(2 ** 20, 64, H, 1), _m(2 ** 20, 16, H, 2)
        return lambda: lib.affine(w, x, save=True)
    if name == "update, one part":
        g = _m(2 ** 20, 130, B, 9)
        return lambda: lib.orthogonalize(g, 1)
    g = _m(2000, 2300, F32, 10)   # update, two parts
    return lambda: lib.orthogonalize(g, 2)


NAMES = ["gated, few columns", "gated, many columns", "gated, gradient", "affine, few columns", "update, one part", "update, two parts"]


def _list(out):
    return list(out) if isinstance(out, tuple) else [out]


def _expire(lib, call):
    """The status of the call after one whose wait ran out (one try does it, as good as always)."""
    for _ in range(50):
        with option(lib, lib.CR_OPT_WAIT_LIMIT_US, 0):
            call()   # returns normally: its waits are the next call's to report
        torch.cuda.synchronize()
        try:
            call()
        except lib.CrError as e:
            return e.name
        torch.cuda.synchronize()
    return "none reported"


@pytest.mark.parametrize("name", NAMES)
def test_an_expired_wait_is_reported_once(lib, name):
    call = _call(lib, name)
    want = [t.clone() for t in _list(call())]
    torch.cuda.synchronize()
    for _ in range(5):
        assert _expire(lib, call) == "CR_ERR_TIMEOUT"
        for _ in range(2):
            for a, b in zip(_list(call()), want):
                assert torch.equal(a, b)
        torch.cuda.synchronize()
