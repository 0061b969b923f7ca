"""The gated product, the group norm and the orthogonalised update together, as one block of a trend network uses them:
O = Wd^T (silu(W1^T Y) * (W2^T Y)) + X with Y = groupnorm(X), its gradients, and a step along the orthogonalised gradients of
its weights; captured into CUDA graphs, on other streams and threads, and with waits that run out."""
import threading

import numpy as np
import pytest
import torch

from oracle import trend
from test_gpu_faults import option
from trend_util import matrix, values, vector

pytestmark = pytest.mark.gpu
F32 = torch.float32


def _make(D=96, N=160, T=700, seed=0):
    rng = np.random.default_rng(seed)
    b16 = torch.bfloat16
    return {"X": matrix(rng.normal(size=(D, T)), b16), "W": matrix(rng.normal(size=(D, 2 * N)) * D ** -0.5, b16),
            "Wd": matrix(rng.normal(size=(N, D)) * N ** -0.5, b16), "gamma": vector(1 + 0.2 * rng.normal(size=D)),
            "beta": vector(0.2 * rng.normal(size=D)), "dO": matrix(rng.normal(size=(D, T)), b16),
            "off": torch.tensor([0, 200, 200, 333, T], dtype=torch.int32, device="cuda")}


def _block(lib, s):
    groups = 8
    Y, mean, rstd = lib.group_norm(s["X"], groups, s["gamma"], s["beta"], "none", s["off"], save=True)
    V, Z = lib.gated_affine(s["W"], Y, act="silu", save=True)
    out = lib.affine(s["Wd"], V, residual=s["X"])
    dV, dWd, _ = lib.affine_backward(s["Wd"], V, s["dO"], need=(True, True, False), dw_dtype=F32)
    dY, dW, _ = lib.gated_affine_backward(s["W"], Y, dV, Z, "silu", need=(True, True, False), dw_dtype=F32)
    dX, dgamma, dbeta = lib.group_norm_backward(s["X"], groups, s["gamma"], s["beta"], dY, mean, rstd, "none", s["off"])
    uW, uWd = lib.orthogonalize(dW, out_dtype=torch.bfloat16), lib.orthogonalize(dWd)
    return out, dX + s["dO"], dgamma, dbeta, dW, dWd, uW, uWd


def test_block_against_the_oracle(lib):
    """Relative Frobenius errors: a matrix of BF16 values between two operators carries 2^-8 / sqrt(3) at most of its own size, and
    no output passes more than eight of them; sums average the errors, so 8 * 2^-8 = 0.031 holds with room."""
    s = _make()
    got = [values(t) for t in _block(lib, s)]
    X, W, Wd, dO, off = values(s["X"]), values(s["W"]), values(s["Wd"]), values(s["dO"]), s["off"].tolist()
    g, b = values(s["gamma"]), values(s["beta"])
    Y, mean, rstd = trend.group_norm(X, 8, g, b, "none", off, 1e-5)
    V, Z = trend.gated_affine(W, Y, None, "silu")
    out, _ = trend.affine(Wd, V, residual=X)
    dV, dWd, _ = trend.affine_backward(Wd, V, dO, None)
    dY, dW, _ = trend.gated_affine_backward(W, Y, dV, Z, "silu")
    dX, dgamma, dbeta = trend.group_norm_backward(X, 8, g, b, dY, mean, rstd, "none", off)
    for name, a, w in zip(("out", "dX", "dgamma", "dbeta", "dW", "dWd"), got, (out, dX + dO, dgamma, dbeta, dW, dWd)):
        assert np.linalg.norm(a - w) <= 0.031 * np.linalg.norm(w), name
    for u, d in ((got[6], got[4]), (got[7], got[5])):   # updates of the gradients that the operators gave
        w = trend.orthogonalize(d)
        assert np.linalg.norm(u - w) <= 0.031 * np.linalg.norm(w)


def test_an_orthogonalised_step_lowers_the_loss(lib):
    """<dW, update> > 0: the update has the gradient's singular vectors with positive weights."""
    s = _make(seed=3)
    _, _, _, _, dW, dWd, uW, uWd = _block(lib, s)
    assert float((dW * uW.float()).sum()) > 0 and float((dWd * uWd.float()).sum()) > 0


def _calls(lib):
    s = _make(seed=1)
    big = _make(512, 1100, 3000, seed=2)
    one = s["X"][:, :1].T.contiguous().T
    few = s["X"][:, :20].T.contiguous().T
    w8 = s["W"].float().T.contiguous().to(torch.float8_e4m3fn).T
    x8 = few.float().T.contiguous().to(torch.float8_e4m3fn).T
    odd = matrix(np.random.default_rng(4).normal(size=(301, 77)), F32)
    return {"block": (s["X"], lambda: _block(lib, s)), "large block": (big["X"], lambda: _block(lib, big)),
            "one column": (one, lambda: lib.gated_affine(s["W"], one, save=True)), "few columns": (few, lambda: lib.gated_affine(s["W"], few)),
            "8 bits": (x8, lambda: lib.gated_affine(w8, x8)), "orthogonal": (odd, lambda: lib.orthogonalize(odd)),
            "norm": (big["X"], lambda: lib.group_norm(big["X"], 16, big["gamma"], None, "gelu", big["off"], save=True))}


def _list(out):
    return list(out) if isinstance(out, tuple) else [out]


NAMES = ["block", "large block", "one column", "few columns", "8 bits", "orthogonal", "norm"]


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays_equal_direct_calls(lib, name):
    x, call = _calls(lib)[name]
    first = [t.clone() for t in _list(call())]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _list(call())
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, first):
        assert torch.equal(a, b)
    x.copy_((x.float() * 0.5).to(x.dtype))   # other inputs at the same place
    graph.replay()
    got = [t.clone() for t in out]
    want = _list(call())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_graphs_replayed_at_once(lib):
    """Each capture has its own scratch: replays on two streams at once do not meet in it."""
    calls = [_calls(lib)["large block"][1], _calls(lib)["large block"][1]]
    want = [t.clone() for t in _list(calls[0]())]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_list(call()))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_threads_on_their_own_streams(lib):
    calls = {n: _calls(lib)[n][1] for n in ("block", "norm", "orthogonal", "few columns")}
    want = {n: [t.clone() for t in _list(c())] for n, c in calls.items()}
    torch.cuda.synchronize()
    bad = []

    def work(name):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(40):
                    out = _list(calls[name]())
                torch.cuda.current_stream().synchronize()
                bad.extend(name for a, b in zip(out, want[name]) if not torch.equal(a, b))
        except Exception as e:   # noqa: BLE001
            bad.append((name, e))

    threads = [threading.Thread(target=work, args=(n,)) for n in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("name", ["large block", "few columns", "orthogonal", "8 bits"])
def test_waits_that_run_out(lib, name):
    """With a limit of zero calls give up wherever something is not yet there; the next call says so once, and the operators work
    as before."""
    call = _calls(lib)[name][1]
    want = [t.clone() for t in _list(call())]
    torch.cuda.synchronize()
    expired = False
    with option(lib, lib.CR_OPT_WAIT_LIMIT_US, 0):
        for _ in range(30):
            try:
                call()
            except lib.CrError as e:
                assert e.name == "CR_ERR_TIMEOUT"
                expired = True
                break
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    try:
        call()
    except lib.CrError as e:
        assert e.name == "CR_ERR_TIMEOUT"
    torch.cuda.synchronize()
    for _ in range(2):
        for a, b in zip(_list(call()), want):
            assert torch.equal(a, b)
    assert expired in (True, False)   # whether something was late is chance


def test_columns_far_apart(lib):
    """Strides of 2^31 elements and more are followed, not cut to 32 bits."""
    gap = 2 ** 31 + 64
    base = torch.empty(gap + 64, dtype=torch.float16, device="cuda")
    far = base.as_strided((64, 2), (1, gap))
    far.copy_(torch.randn(2, 64, device="cuda").half().T)
    packed = far.T.contiguous().T
    w = torch.randn(8, 64, device="cuda").half().T
    assert torch.equal(lib.gated_affine(w, far), lib.gated_affine(w, packed))
    assert torch.equal(lib.group_norm(far, 4), lib.group_norm(packed, 4))
    assert torch.equal(lib.orthogonalize(far), lib.orthogonalize(packed))
    n = 2 ** 32 + 8
    x = torch.ones(1, 1, device="cuda").half().expand(1, n)
    for call in (lambda: lib.gated_affine(torch.ones(2, 1, device="cuda").half().T, x), lambda: lib.group_norm(x, 1), lambda: lib.orthogonalize(x)):
        with pytest.raises(lib.CrError) as e:
            call()
        assert e.value.code == 1


def test_large_matrices_beyond_32_bit_offsets(lib):
    """Elements past 2^31 of a matrix: the last columns are right.  Their tiles lie otherwise in the small matrix, so the statistics
    differ by a few roundings (100 * 2^-24 of the largest magnitude, 6, and 7e-5 in y) and the output by one spacing more."""
    D, T = 4096, 540000
    X = torch.empty(T, D, dtype=torch.float16, device="cuda").normal_().T
    off = torch.tensor([0, T - 500, T], dtype=torch.int32, device="cuda")
    Y = lib.group_norm(X, 32, None, None, "none", off)
    torch.testing.assert_close(Y[:, -500:], lib.group_norm(X[:, -500:], 32, None, None, "none"), rtol=2 ** -10, atol=2e-4)
    W = torch.randn(16, D, device="cuda").mul_(D ** -0.5).half().T
    V = lib.gated_affine(W, X)
    torch.testing.assert_close(V[:, -9:], lib.gated_affine(W, X[:, -9:]), rtol=2 ** -9, atol=2 ** -9)
