"""Measured cases of the trend-network operators: the affine product with its epilogue, the
root-mean-square norm with the residual and an 8-bit output, and the gated recurrence.

Matrices are features x columns and column-major, like the rest of the package: a column is
one site at one time, and is contiguous in memory.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100
EPS = 1e-6
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def listed():
    return [
        # one site answered at one time step: latency and the read of the weights
        {"name": "affine one column", "op": "affine", "K": 2048, "N": 2048, "M": 1, "type": "bf16", "act": "silu",
         "bias": True, "residual": False},
        # a few sites at one time step: the weights streamed once for sixteen columns
        {"name": "affine few columns", "op": "affine", "K": 4096, "N": 12288, "M": 16, "type": "f16", "act": "none",
         "bias": True, "residual": True},
        # a ragged batch of sites, between the streaming and the compute-bound ends
        {"name": "affine ragged batch", "op": "affine", "K": 2048, "N": 8192, "M": 1537, "type": "f16", "act": "gelu",
         "bias": True, "residual": False},
        # answering a full grid in 8 bits
        {"name": "affine 8 bits", "op": "affine", "K": 4096, "N": 8192, "M": 8192, "type": "e4m3", "act": "none",
         "bias": True, "residual": True},
        # the widest layer over a full grid
        {"name": "affine largest", "op": "affine", "K": 4096, "N": 16384, "M": 8192, "type": "bf16", "act": "silu",
         "bias": True, "residual": False},
        # one training step's gradients on a ragged batch
        {"name": "affine backward", "op": "affine_backward", "K": 2048, "N": 8192, "M": 4099, "type": "bf16",
         "act": "silu"},
        # normalising four columns before an 8-bit product: latency
        {"name": "norm four columns", "op": "norm", "D": 4096, "T": 4, "type": "f16", "out": "e4m3", "residual": True},
        # the same over a grid's whole history
        {"name": "norm long", "op": "norm", "D": 4096, "T": 32768, "type": "bf16", "out": "e4m3", "residual": True},
        # training, at a width that is no power of two and an odd number of columns
        {"name": "norm backward", "op": "norm_backward", "D": 2560, "T": 16411, "type": "bf16", "residual": True},
        # one long series
        {"name": "scan long", "op": "scan", "D": 2048, "T": 65536, "seqs": 1, "type": "bf16", "gate": "convex"},
        # a training step over ragged series, some of them empty
        {"name": "scan training", "op": "scan_training", "D": 1536, "T": 50021, "seqs": 77, "type": "f16",
         "gate": "variance"},
        # one time step of 64 series
        {"name": "scan step", "op": "step", "D": 4096, "B": 64, "type": "bf16", "gate": "convex"},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["affine", "affine", "affine", "affine_backward", "norm", "norm_backward", "scan", "scan_training", "step"])
    half = rng.choice(["f16", "bf16"])
    if op in ("affine", "affine_backward"):
        while True:
            k, n = _log_int(rng, 256, 8192), _log_int(rng, 256, 16384)
            m = _log_int(rng, 1, 8192) if op == "affine" else _log_int(rng, 64, 8192)
            if rng.random() < 0.75:   # widths are multiples of 16 in most programs
                k, n = -(-k // 16) * 16, -(-n // 16) * 16
            if k * n * m <= 4096 * 16384 * 8192 // (1 if op == "affine" else 2):
                break
        act = rng.choice(["none", "relu", "silu", "gelu"])
        if op == "affine_backward":
            return {"op": op, "K": k, "N": n, "M": m, "type": half, "act": act}
        return {"op": op, "K": k, "N": n, "M": m, "type": rng.choice([half, half, "e4m3"]), "act": act,
                "bias": rng.random() < 0.7, "residual": rng.random() < 0.5}
    if op in ("norm", "norm_backward"):
        while True:
            d, t = _log_int(rng, 64, 16384), _log_int(rng, 1, 65536)
            if rng.random() < 0.75:
                d = -(-d // 16) * 16
            if d * t <= 4096 * 32768:
                break
        c = {"op": op, "D": d, "T": t, "type": half, "residual": rng.random() < 0.6}
        if op == "norm":
            c["out"] = rng.choice(["e4m3", half])
        return c
    gate = rng.choice(["coeff", "convex", "variance"])
    kind = rng.choice([half, half, "f32"])
    if op == "step":
        d = _log_int(rng, 64, 8192)
        return {"op": op, "D": d if rng.random() < 0.25 else -(-d // 8) * 8, "B": _log_int(rng, 1, 4096), "type": kind,
                "gate": gate}
    while True:
        d, t = _log_int(rng, 64, 8192), _log_int(rng, 16, 131072)
        if rng.random() < 0.75:
            d = -(-d // 8) * 8
        if d * t * (2 if kind == "f32" else 1) <= 2048 * 65536 // (1 if op == "scan" else 2):
            break
    return {"op": op, "D": d, "T": t, "seqs": min(t, _log_int(rng, 1, 512)), "type": kind, "gate": gate}


# ---------------------------------------------------------------- inputs

def _normal(gen, rows, cols, kind, scale=1.0, shift=0.0):
    """A rows x cols column-major matrix of normal values."""
    x = torch.randn((cols, rows), generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(scale).add_(shift).to(TYPES[kind]).T


def _eight_bits(x):
    """x (rows x cols, column-major) as e4m3 with a scale per column."""
    s = x.abs().amax(0).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (x / s).T.to(torch.float8_e4m3fn).T, s


def _offsets(case, seed):
    """Ends of the packed series: random cuts, so that some series are short or empty."""
    gen = torch.Generator().manual_seed(seed)
    t, n = case["T"], case["seqs"]
    cuts = torch.randint(0, t + 1, (n - 1,), generator=gen).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([t])]).to(torch.int32).cuda()


def _gates(gen, case, rows, cols):
    if case["gate"] == "coeff":   # coefficients between 0.5 and 1
        g = torch.rand((cols, rows), generator=gen, device="cuda").mul_(0.5).add_(0.5)
        return g.to(TYPES[case["type"]]).T
    return _normal(gen, rows, cols, case["type"], 1.5, 2.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, kind = case["op"], case["type"]
    s = {"case": case}
    if op in ("affine", "affine_backward"):
        k, n, m = case["K"], case["N"], case["M"]
        if kind == "e4m3":
            s["W"], s["ws"] = _eight_bits(_normal(gen, k, n, "f32", k ** -0.5))
            s["X"], s["xs"] = _eight_bits(_normal(gen, k, m, "f32"))
        else:
            s["W"], s["ws"] = _normal(gen, k, n, kind, k ** -0.5), None
            s["X"], s["xs"] = _normal(gen, k, m, kind), None
        half = "bf16" if kind == "e4m3" else kind
        s["out"] = TYPES[half]
        if op == "affine":
            s["b"] = torch.randn(n, generator=gen, device="cuda").mul_(0.5) if case["bias"] else None
            s["R"] = _normal(gen, n, m, half) if case["residual"] else None
        else:
            z = s["X"].T.float() @ s["W"].float()
            z += torch.randn(n, generator=gen, device="cuda").mul_(0.5)
            s["Z"] = z.to(TYPES[kind]).T
            s["dY"] = _normal(gen, n, m, kind)
    elif op in ("norm", "norm_backward"):
        d, t = case["D"], case["T"]
        s["gamma"] = torch.randn(d, generator=gen, device="cuda").mul_(0.1).add_(1.0)
        s["X"] = _normal(gen, d, t, kind, 2.0)
        s["R"] = _normal(gen, d, t, kind) if case["residual"] else None
        if op == "norm_backward":
            s["dY"] = _normal(gen, d, t, kind)
    elif op in ("scan", "scan_training"):
        d, t = case["D"], case["T"]
        s["G"], s["X"] = _gates(gen, case, d, t), _normal(gen, d, t, kind)
        s["off"] = _offsets(case, seed)
        s["h0"] = _normal(gen, d, case["seqs"], "f32")
        if op == "scan_training":
            s["dH"] = _normal(gen, d, t, kind)
            s["dhT"] = _normal(gen, d, case["seqs"], "f32")
    else:
        d, b = case["D"], case["B"]
        s["G"], s["X"], s["h"] = _gates(gen, case, d, b), _normal(gen, d, b, kind), _normal(gen, d, b, "f32")
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _activation(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(z)


def _plain_affine(s):
    z = s["X"].T.float() @ s["W"].float()
    if s["ws"] is not None:
        z = z * s["ws"] * s["xs"][:, None]
    if s["b"] is not None:
        z = z + s["b"]
    y = _activation(z, s["case"]["act"])
    if s["R"] is not None:
        y = y + s["R"].T.float()
    return y.to(s["out"]).T


def _plain_affine_backward(s):
    g = s["dY"].T.float() * _slope(s["Z"].T.float(), s["case"]["act"])
    dx = g @ s["W"].T.float()
    dw = g.T @ s["X"].T.float()
    return dx.to(s["out"]).T, dw.to(s["out"]).T, g.sum(0)


def _plain_norm(s):
    h = s["X"].T.float()
    if s["R"] is not None:
        h = h + s["R"].T.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"]
    kept = h.to(s["X"].dtype).T if s["R"] is not None else None
    if s["case"]["out"] != "e4m3":
        return y.to(s["X"].dtype).T, kept
    scale = y.abs().amax(1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (y / scale[:, None]).to(torch.float8_e4m3fn).T, scale, kept


def _plain_norm_backward(s):
    h, dy = s["X"].T.float(), s["dY"].T.float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    u = dy * s["gamma"]
    dx = r * u - h * (r * r * r * (u * h).mean(1, keepdim=True))
    if s["R"] is not None:   # the gradient that arrives at H past the norm
        dx = dx + s["R"].T.float()
    return dx.to(s["X"].dtype).T, (dy * h * r).sum(0)


def _coefficients(g, gate):
    """(a, c) of h = a h' + c x."""
    if gate == "coeff":
        return g, torch.ones_like(g)
    a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    return a, rest if gate == "convex" else torch.sqrt(rest * (1.0 + a))


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t for all rows t: each round doubles the span that b_t covers."""
    span = 1
    while span < a.shape[0]:
        b = torch.cat([b[:span], b[span:] + a[span:] * b[:-span]])
        a = torch.cat([a[:span], a[span:] * a[:-span]])
        span *= 2
    return b


def _plain_scan(s):
    """(h, the state before each row, a, c, hT, first rows, last rows, nonempty series), rows = time."""
    a, c = _coefficients(s["G"].T.float(), s["case"]["gate"])
    off = s["off"].long()
    full = (off[1:] > off[:-1]).nonzero()[:, 0]
    first, last = off[:-1][full], off[1:][full] - 1
    h0 = s["h0"].T
    cut, b = a.clone(), c * s["X"].T.float()
    b[first] += a[first] * h0[full]
    cut[first] = 0.0
    h = _doubling(cut, b)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[first] = h0[full]
    end = h0.clone()
    end[full] = h[last]
    return h, before, a, c, end, first, last, full


def _plain_scan_training(s):
    h, before, a, c, end, first, last, full = _plain_scan(s)
    kind, gate = s["X"].dtype, s["case"]["gate"]
    d = s["dH"].T.float()
    d[last] += s["dhT"].T[full]
    follow = torch.cat([a[1:], torch.zeros_like(a[:1])])
    follow[last] = 0.0
    q = _doubling(follow.flip(0), d.flip(0)).flip(0)
    dh0 = s["dhT"].T.clone()
    dh0[full] = a[first] * q[first]
    x = s["X"].T.float()
    if gate == "coeff":
        dg = q * before
    elif gate == "convex":
        dg = q * (before - x) * (a * c)
    else:
        rest = torch.sigmoid(-s["G"].T.float())
        dg = q * a * (before * rest - x * a * torch.sqrt(rest / (1.0 + a)))
    return h.to(kind).T, end.T, dg.to(kind).T, (q * c).to(kind).T, dh0.T


def _plain_step(s):
    a, c = _coefficients(s["G"].T.float(), s["case"]["gate"])
    h = a * s["h"].T + c * s["X"].T.float()
    return h.to(s["X"].dtype).T, h.T


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "scan":
            h, _, _, _, end, _, _, _ = _plain_scan(s)
            return h.to(s["X"].dtype).T, end.T
        return {"affine": _plain_affine, "affine_backward": _plain_affine_backward, "norm": _plain_norm,
                "norm_backward": _plain_norm_backward, "scan_training": _plain_scan_training, "step": _plain_step}[op](s)
    import mixed_precision_dense_mat_gb300 as cr
    if op == "affine":
        return cr.affine(s["W"], s["X"], s["b"], c["act"], s["R"], w_scale=s["ws"], x_scale=s["xs"], out_dtype=s["out"])
    if op == "affine_backward":
        return cr.affine_backward(s["W"], s["X"], s["dY"], s["Z"], c["act"])
    if op == "norm":
        if c["out"] == "e4m3":
            return cr.rmsnorm_e4m3(s["X"], s["gamma"], s["R"], eps=EPS)
        return cr.rmsnorm(s["X"], s["gamma"], s["R"], eps=EPS)
    if op == "norm_backward":
        return cr.rmsnorm_backward(s["X"], s["gamma"], s["dY"], s["R"], eps=EPS)
    if op == "scan":
        return cr.gated_scan(s["G"], s["X"], c["gate"], s["off"], s["h0"])
    if op == "scan_training":
        h, end, saved = cr.gated_scan(s["G"], s["X"], c["gate"], s["off"], s["h0"], save=True)
        dg, dx, dh0 = cr.gated_scan_backward(s["G"], s["X"], s["dH"], c["gate"], s["off"], s["h0"], s["dhT"], saved)
        return h, end, dg, dx, dh0
    return cr.gated_step(s["G"], s["X"], s["h"], c["gate"])


def work(case):
    op, e = case["op"], SIZE[case["type"]]
    if op in ("affine", "affine_backward"):
        k, n, m = case["K"], case["N"], case["M"]
        if op == "affine_backward":
            return {"bytes": 2 * (2 * k * n + 2 * k * m + n * m * (1 if case["act"] == "none" else 2)) + 4 * n,
                    "flops": 4 * k * n * m}
        extra = (4 * n if case["bias"] else 0) + (4 * (n + m) if case["type"] == "e4m3" else 0)
        return {"bytes": e * (k * n + k * m) + 2 * n * m * (2 if case["residual"] else 1) + extra,
                "flops": 2 * k * n * m}
    if op == "norm":
        d, t = case["D"], case["T"]
        per = e + (1 if case["out"] == "e4m3" else e) + (2 * e if case["residual"] else 0)
        return {"bytes": d * t * per + 4 * d + (4 * t if case["out"] == "e4m3" else 0), "flops": 6 * d * t}
    if op == "norm_backward":
        d, t = case["D"], case["T"]
        return {"bytes": d * t * e * (4 if case["residual"] else 3) + 8 * d, "flops": 12 * d * t}
    d = case["D"]
    if op == "step":
        return {"bytes": d * case["B"] * (3 * e + 8), "flops": 8 * d * case["B"]}
    t, n = case["T"], case["seqs"]
    if op == "scan":
        return {"bytes": 3 * e * d * t + 8 * d * n, "flops": 8 * d * t}
    return {"bytes": 6 * e * d * t + 16 * d * n, "flops": 24 * d * t}


# ---------------------------------------------------------------- the definitions in 64 bits

def _sigmoid64(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * _sigmoid64(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    return z


def _dact64(z, act):
    if act == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act == "silu":
        p = _sigmoid64(z)
        return p + z * p * _sigmoid64(-z)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(z)


def _exact_affine(s):
    w, x = s["W"].double(), s["X"].double()
    if s["ws"] is not None:
        w, x = w * s["ws"].double()[None, :], x * s["xs"].double()[None, :]
    z = w.T @ x
    if s["b"] is not None:
        z = z + s["b"].double()[:, None]
    y = _act64(z, s["case"]["act"])
    return y if s["R"] is None else y + s["R"].double()


def _exact_affine_backward(s):
    g = s["dY"].double() * _dact64(s["Z"].double(), s["case"]["act"])
    return s["W"].double() @ g, s["X"].double() @ g.T, g.sum(1)


def _exact_norm(s):
    h = s["X"].double()
    if s["R"] is not None:
        h = h + s["R"].double()
    y = s["gamma"].double()[:, None] * h / torch.sqrt((h ** 2).mean(0) + EPS)
    kept = h if s["R"] is not None else None
    if s["case"]["out"] != "e4m3":
        return y, kept
    scale = torch.clamp(y.abs().max(0).values, min=AMAX_FLOOR) / E4M3_MAX
    return y / scale, scale, kept


def _exact_norm_backward(s):
    h, dy, gamma = s["X"].double(), s["dY"].double(), s["gamma"].double()[:, None]
    root = torch.sqrt((h ** 2).mean(0) + EPS)
    n = h / root
    u = gamma * dy
    dx = (u - n * (u * n).mean(0)) / root
    if s["R"] is not None:
        dx = dx + s["R"].double()
    return dx, (dy * n).sum(1)


def _exact_gate(g, gate):
    """(a, c, da/dg, dc/dg) in 64 bits."""
    if gate == "coeff":
        return g, torch.ones_like(g), torch.ones_like(g), torch.zeros_like(g)
    a, r = _sigmoid64(g), _sigmoid64(-g)
    if gate == "convex":
        return a, r, a * r, -a * r
    c = torch.sqrt(1.0 - a * a)
    return a, c, a * r, -a * (a * r) / c


def _exact_scan(s, backward):
    """Step by step along each series."""
    g, x = s["G"].T.double(), s["X"].T.double()
    a, c, da, dc = _exact_gate(g, s["case"]["gate"])
    b, off = c * x, s["off"].tolist()
    h, before, end = torch.empty_like(b), torch.empty_like(b), s["h0"].T.double().clone()
    for i in range(len(off) - 1):
        state = end[i]
        for t in range(off[i], off[i + 1]):
            before[t] = state
            state = torch.addcmul(b[t], a[t], state, out=h[t])
        end[i] = state
    if not backward:
        return h.T, end.T
    q, dh0 = s["dH"].T.double(), s["dhT"].T.double().clone()
    for i in range(len(off) - 1):
        carry = dh0[i]
        for t in range(off[i + 1] - 1, off[i] - 1, -1):
            q[t] += carry
            carry = a[t] * q[t]
        dh0[i] = carry
    return h.T, end.T, (q * (before * da + x * dc)).T, (q * c).T, dh0.T


def _exact_step(s):
    a, c, _, _ = _exact_gate(s["G"].double(), s["case"]["gate"])
    h = a * s["h"].double() + c * s["X"].double()
    return h, h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan" or op == "scan_training":
        return _exact_scan(s, op == "scan_training")
    return {"affine": _exact_affine, "affine_backward": _exact_affine_backward, "norm": _exact_norm,
            "norm_backward": _exact_norm_backward, "step": _exact_step}[op](s)
