"""Bounded waits of the trend-network operators: with a limit of zero (CR_OPT_WAIT_LIMIT_US) they give up wherever
they find something not yet there.  The calls end, the next one reports it once, and the operators work as before."""
import pytest
import torch

from test_gpu_faults import option

pytestmark = pytest.mark.gpu


def _list(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def _expire(lib, call, tries=50):
    """Whether a call with a zero limit was reported as expired by the one after it."""
    with option(lib, lib.CR_OPT_WAIT_LIMIT_US, 0):
        for _ in range(tries):
            try:
                call()
            except lib.CrError as e:
                assert e.name == "CR_ERR_TIMEOUT"
                return True
            torch.cuda.synchronize()
    return False


def _check(lib, call, surely=True):
    want = [t.clone() for t in _list(call())]
    torch.cuda.synchronize()
    expired = _expire(lib, call)
    assert expired or not surely
    if not expired:   # nothing left to report, or the last try's
        try:
            call()
        except lib.CrError as e:
            assert e.name == "CR_ERR_TIMEOUT"
    assert lib.get_option(lib.CR_OPT_WAIT_LIMIT_US) == 2000000
    for _ in range(2):
        for a, b in zip(_list(call()), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [304, 301])   # by TMA, and without it
def test_recurrence(lib, kind, D):
    """Chunks that wait for earlier ones: some of the thousands are never there at once."""
    T = 30000
    g, x = torch.randn(T, D, device="cuda").to(kind).T, torch.randn(T, D, device="cuda").to(kind).T
    off = torch.tensor([0, 11000, 11000, T], dtype=torch.int32, device="cuda")
    _check(lib, lambda: lib.gated_scan(g, x, "convex", off, save=True))
    saved = lib.gated_scan(g, x, "convex", off, save=True)[2]
    _check(lib, lambda: lib.gated_scan_backward(g, x, x, "convex", off, saved=saved))


@pytest.mark.parametrize("D", [512, 768, 4096, 10240])
def test_norm(lib, D):
    """Copies into shared memory: whether they are there at once is chance."""
    T = 3000
    x, d, g = torch.randn(T, D, device="cuda").half().T, torch.randn(T, D, device="cuda").half().T, torch.rand(D, device="cuda")
    _check(lib, lambda: lib.rmsnorm(x, g, d), surely=False)
    _check(lib, lambda: lib.rmsnorm_e4m3(x, g), surely=False)
    _check(lib, lambda: lib.rmsnorm_backward(x, g, d, x), surely=False)


@pytest.mark.parametrize("K,N,M", [(4096, 2048, 16), (1024, 512, 60), (200, 300, 100), (515, 300, 7)])
def test_affine_few_columns(lib, K, N, M):
    """Copies, products and, between the CTAs of a cluster, partial sums: whether they are there at once is chance."""
    w, x = torch.randn(N, K, device="cuda").half().T, torch.randn(M, K, device="cuda").half().T
    b, r = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").half().T
    _check(lib, lambda: lib.affine(w, x, b, "silu", r, save=True), surely=False)


@pytest.mark.parametrize("K,N,M", [(1024, 2048, 1500), (64, 4096, 3000), (3000, 520, 700)])
def test_affine_many_columns(lib, K, N, M):
    """Pairs of CTAs: operands, products, residuals and outputs in flight when a warp gives up."""
    w, x = torch.randn(N, K, device="cuda").half().T, torch.randn(M, K, device="cuda").half().T
    b, r = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").half().T
    _check(lib, lambda: lib.affine(w, x, b, "silu", r), surely=False)
    _check(lib, lambda: lib.affine(w, x, b, "silu", r, save=True), surely=False)
    _check(lib, lambda: lib.affine(w, x, out_dtype=torch.float32), surely=False)
    _check(lib, lambda: lib.affine_backward(w, x, r, r, "gelu"), surely=False)


@pytest.mark.parametrize("reports", ["step", "long norm", "long norm backward"])
def test_calls_without_waits_report_too(lib, reports):
    g, x = torch.randn(30000, 304, device="cuda").T, torch.randn(30000, 304, device="cuda").T
    y, c = torch.randn(2, 17000, device="cuda").T, torch.ones(17000, device="cuda")
    call = {"step": lambda: lib.gated_step(x[:, :3], x[:, :3], g[:, :3]), "long norm": lambda: lib.rmsnorm(y, c),
            "long norm backward": lambda: lib.rmsnorm_backward(y, c, y)}[reports]
    lib.gated_scan(g, x)
    call()
    for _ in range(50):
        with option(lib, lib.CR_OPT_WAIT_LIMIT_US, 0):
            lib.gated_scan(g, x)
        torch.cuda.synchronize()
        try:
            call()
        except lib.CrError as e:
            assert e.name == "CR_ERR_TIMEOUT"
            break
    else:
        raise AssertionError("no call reported the recurrence's wait")
    call()
    lib.gated_scan(g, x)
