"""The wait word of the trend-network operators (a device-side wait that ran out is reported by the next call, once, and that call
does none of its work): gradients of the products, whatever is wanted of them."""
import pytest
import torch

from test_gpu_faults import option

pytestmark = pytest.mark.gpu
F16 = 1


def _expire(lib):
    """Leaves the report of a recurrence's expired wait behind: some of thousands of chunks are never there at once."""
    g, x = torch.randn(30000, 304, device="cuda").T, torch.randn(30000, 304, device="cuda").T
    lib.gated_scan(g, x)
    torch.cuda.synchronize()

    def once():
        with option(lib, lib.CR_OPT_WAIT_LIMIT_US, 0):
            lib.gated_scan(g, x)
        torch.cuda.synchronize()
    return once


def _calls(lib, gated, K=96, N=64, M=520):
    """call(dX, dW, db wanted) -> (status, outputs), which hold 3 beforehand."""
    half = torch.float16
    rows = 2 * N if gated else N
    W, X = torch.randn(rows, K, device="cuda").to(half), torch.randn(M, K, device="cuda").to(half)
    dY, Z = torch.randn(M, N, device="cuda").to(half), torch.randn(M, rows, device="cuda").to(half)

    def call(need):
        shapes = ((M, K, half), (rows, K, half), (rows, 1, torch.float32))
        outs = [torch.full((a, b), 3.0, dtype=t, device="cuda") for a, b, t in shapes]
        p = [o.data_ptr() if n else None for o, n in zip(outs, need)]
        f = lib._lib.cr_gated_affine_backward if gated else lib._lib.cr_affine_backward
        code = f(F16, W.data_ptr(), K, X.data_ptr(), K, dY.data_ptr(), N, Z.data_ptr(), rows, K, N, M, 2, p[0], K, F16, p[1], K, p[2],
                 torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        return lib.STATUS[code] if code else "CR_OK", outs
    return call


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("need", [(0, 0, 1), (1, 0, 0), (0, 1, 0), (1, 1, 1), (1, 1, 0)])
def test_gradients_report_before_any_work(lib, gated, need):
    once, call = _expire(lib), _calls(lib, gated)
    status, want = call(need)
    assert status == "CR_OK"
    assert all(bool((o == 3.0).all()) != bool(n) for o, n in zip(want, need))
    for _ in range(50):
        once()
        status, outs = call(need)
        if status != "CR_OK":
            break
    assert status == "CR_ERR_TIMEOUT"
    assert all(bool((o == 3.0).all()) for o in outs)
    status, outs = call(need)
    assert status == "CR_OK" and all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("gated", [False, True])
def test_nothing_wanted_is_no_call(lib, gated):
    """It has nothing to do, and leaves the report to the next call."""
    once, call = _expire(lib), _calls(lib, gated)
    for _ in range(50):
        once()
        assert call((0, 0, 0))[0] == "CR_OK"
        status = call((0, 0, 1))[0]
        if status != "CR_OK":
            break
    assert status == "CR_ERR_TIMEOUT"
    assert call((1, 1, 1))[0] == "CR_OK"
