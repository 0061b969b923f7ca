"""The trend-network operators called by several host threads at once, on streams of their own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_norms_of_different_widths_in_two_threads(lib):
    """The same kernel with different amounts of shared memory: neither call may lose its share to the other.
    Straight calls of the C entries, so that the threads meet inside them."""
    T, failures, results = 200, [], {}
    inputs = {D: (torch.randn(T, D, device="cuda"), torch.ones(D, device="cuda")) for D in (1032, 4096)}
    want = {D: (lib.rmsnorm(x.T, g)[0].T, *lib.rmsnorm_backward(x.T, g, x.T)) for D, (x, g) in inputs.items()}
    torch.cuda.synchronize()

    def work(D):
        x, g = inputs[D]
        y, dx, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(g)
        s = torch.cuda.Stream()
        px, pg = x.data_ptr(), g.data_ptr()
        forward = (0, px, D, None, 0, pg, D, T, 1e-6, None, 0, 0, y.data_ptr(), D, None, s.cuda_stream)
        backward = (0, px, D, pg, px, D, None, 0, D, T, 1e-6, dx.data_ptr(), D, dg.data_ptr(), s.cuda_stream)
        bad = 0
        for _ in range(10000):
            bad += lib._lib.cr_rmsnorm(*forward) != 0
            bad += lib._lib.cr_rmsnorm_backward(*backward) != 0
        s.synchronize()
        if bad:
            failures.append((D, bad, lib._lib.cr_last_error_detail()))
        results[D] = (y, dx, dg)

    threads = [threading.Thread(target=work, args=(D,)) for D in inputs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
    for D in inputs:
        y, dx, dg = results[D]
        assert torch.equal(y, want[D][0]) and torch.equal(dx.T, want[D][1]) and torch.equal(dg, want[D][2])
