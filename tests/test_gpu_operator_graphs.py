"""The trend-network operators captured into CUDA graphs: replays give what direct calls give."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _half(rows, cols, seed, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(cols, rows, device="cuda", generator=gen) * scale).bfloat16().T


def _calls(lib):
    """name -> (inputs, function of them): every kernel of the operators, and chains of them."""
    off = torch.tensor([0, 700, 700, 3000], dtype=torch.int32, device="cuda")

    def block(x, w1, w2, g):   # norm, two products, recurrence, and all their gradients
        y, _ = lib.rmsnorm(x, g)
        a, z = lib.affine(w1, y, None, "silu", save=True)
        s, last, saved = lib.gated_scan(a, a, "convex", off, save=True)
        o = lib.affine(w2, s, residual=x)
        ds, dw2, db2 = lib.affine_backward(w2, s, o)
        dg, da, dh0 = lib.gated_scan_backward(a, a, ds, "convex", off, saved=saved)
        dy, dw1, db1 = lib.affine_backward(w1, y, dg + da, z, "silu")
        dx, dgamma = lib.rmsnorm_backward(x, g, dy, o)
        return y, a, z, s, last, o, dw2, db2, dh0, dw1, db1, dx, dgamma

    def answer(x, w, g, h):   # one time step in 8 bits
        y, scale, _ = lib.rmsnorm_e4m3(x, g)
        w8 = w.float().T.contiguous().to(torch.float8_e4m3fn).T
        v = lib.affine(w8, y, x_scale=scale)
        return y.float(), scale, v, *lib.gated_step(v, v, h)

    gamma = torch.rand(512, device="cuda") + 0.5
    return {
        "one column": ((_half(512, 256, 1, 0.05), _half(512, 1, 2)), lambda w, x: lib.affine(w, x, act="gelu")),
        "few columns": ((_half(2048, 1024, 1, 0.02), _half(2048, 24, 2)), lambda w, x: lib.affine(w, x, act="silu")),
        "many columns": ((_half(512, 2048, 1, 0.05), _half(512, 1500, 2)), lambda w, x: lib.affine(w, x, act="silu", save=True)),
        "unaligned": ((_half(515, 300, 1, 0.05), _half(515, 200, 2)), lambda w, x: lib.affine_backward(w, x, lib.affine(w, x))),
        "gradient": ((_half(768, 2304, 1, 0.04), _half(768, 1100, 2), _half(2304, 1100, 3), _half(2304, 1100, 4)),
                     lambda w, x, dy, z: lib.affine_backward(w, x, dy, z, "silu")),
        "long columns": ((_half(17000, 20, 1), _half(17000, 20, 2), torch.rand(17000, device="cuda")),
                         lambda x, d, g: (*lib.rmsnorm(x, g)[:1], *lib.rmsnorm_backward(x, g, d))),
        "block": ((_half(512, 3000, 1), _half(512, 512, 2, 0.04), _half(512, 512, 3, 0.04), gamma), block),
        "answer": ((_half(512, 40, 1), _half(512, 512, 2, 0.04), gamma, torch.randn(40, 512, device="cuda").T), answer),
    }


NAMES = ["one column", "few columns", "many columns", "unaligned", "gradient", "long columns", "block", "answer"]


def _list(out):
    return list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays_equal_direct_calls(lib, name):
    inputs, call = _calls(lib)[name]
    first = [t.clone() for t in _list(call(*inputs))]   # the first call outside a capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _list(call(*inputs))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, first):
        assert torch.equal(a, b)
    inputs[-1].mul_(0.5)   # other inputs at the same place
    graph.replay()
    got = [t.clone() for t in out]
    want = _list(call(*inputs))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
