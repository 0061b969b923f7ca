"""A learned space-time trend for universal kriging, trained and answered with the trend-network operators.

Every site has a series of covariates.  A small recurrent block turns each series into the site's
trend at the last time,

    A = silu(W1^T x + b1);  Y = rmsnorm(A);  G = Wg^T Y + bg;  V = gelu(Wv^T Y + bv)
    S_t = a_t S_{t-1} + sqrt(1 - a_t^2) V_t,  a = sigmoid(G);  O = Wo^T S + bo + A;  m = Wh^T O_T + bh

is fitted to the observed sites by gradient descent, and m becomes a column of the kriging design next
to the constant and a coordinate.  The next time step is then answered from the kept states, with the
gate and value products in 8 bits.

    python examples/recurrent_trend.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import inputgen                                # noqa: E402
import mixed_precision_dense_mat_gb300 as cr   # noqa: E402

GATE = "variance"


def columns(a):
    """A (rows, columns) array as a column-major BF16 CUDA matrix."""
    return torch.from_numpy(np.ascontiguousarray(a.T)).cuda().bfloat16().T


class RecurrentTrend:
    """The block's parameters: FP32 masters, and the BF16 weights that the products read."""

    def __init__(self, features, width, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(k, n):
            return (torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5).T

        self.master = {"W1": weight(features, width), "Wg": weight(width, width), "Wv": weight(width, width),
                       "Wo": weight(width, width), "Wh": weight(width, 1)}
        for n in ("b1", "bg", "bv", "bo"):
            self.master[n] = torch.zeros(width, device="cuda")
        self.master["bg"] += 2.0   # start with long memories
        self.master["bh"] = torch.zeros(1, device="cuda")
        self.master["gamma"] = torch.ones(width, device="cuda")
        self.update({}, 0.0)

    def update(self, grads, rate):
        """A gradient step, no longer than `rate` times the gradients' norm cut at one."""
        if grads:
            norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads.values()))
            cut = (1.0 / norm.clamp_min(1.0)).float()
        for n, g in grads.items():
            self.master[n] -= rate * cut * g
        self.w = {n: m.T.contiguous().bfloat16().T for n, m in self.master.items() if m.dim() == 2}

    def forward(self, X, offsets, last):
        w, p = self.w, self.master
        A, ZA = cr.affine(w["W1"], X, p["b1"], "silu", save=True)
        Y, _ = cr.rmsnorm(A, p["gamma"])
        G = cr.affine(w["Wg"], Y, p["bg"])
        V, ZV = cr.affine(w["Wv"], Y, p["bv"], "gelu", save=True)
        S, state, saved = cr.gated_scan(G, V, GATE, offsets, save=True)
        O = cr.affine(w["Wo"], S, p["bo"], residual=A)   # noqa: E741
        OL = O.T[last].T
        m = cr.affine(w["Wh"], OL, p["bh"], out_dtype=torch.float32)[0]
        return m, state, (X, offsets, last, A, ZA, Y, G, V, ZV, S, saved, O, OL)

    def gradients(self, dm, kept):
        X, offsets, last, A, ZA, Y, G, V, ZV, S, saved, O, OL = kept   # noqa: E741
        w, f32 = self.w, torch.float32
        dOL, dWh, dbh = cr.affine_backward(w["Wh"], OL, dm[None].bfloat16(), dw_dtype=f32)
        dO = torch.zeros_like(O.T)
        dO[last] = dOL.T
        dO = dO.T
        dS, dWo, dbo = cr.affine_backward(w["Wo"], S, dO, dw_dtype=f32)
        dG, dV, _ = cr.gated_scan_backward(G, V, dS, GATE, offsets, saved=saved)
        dYg, dWg, dbg = cr.affine_backward(w["Wg"], Y, dG, dw_dtype=f32)
        dYv, dWv, dbv = cr.affine_backward(w["Wv"], Y, dV, ZV, "gelu", dw_dtype=f32)
        dA, dgamma = cr.rmsnorm_backward(A, self.master["gamma"], dYg + dYv, dO)
        _, dW1, db1 = cr.affine_backward(w["W1"], X, dA, ZA, "silu", need=(False, True, True), dw_dtype=f32)
        return {"W1": dW1, "Wg": dWg, "Wv": dWv, "Wo": dWo, "Wh": dWh, "b1": db1, "bg": dbg, "bv": dbv, "bo": dbo, "bh": dbh,
                "gamma": dgamma}

    def eight_bits(self):
        """The gate and value weights in e4m3 with a scale per output, laid out once for answering."""
        kept = {}
        for n in ("Wg", "Wv"):
            m = self.master[n]
            s = m.abs().amax(0).clamp_min(1e-30) / 448.0
            kept[n] = ((m / s).T.contiguous().to(torch.float8_e4m3fn).T, s)
        return kept

    def step(self, x, state, weights8=None):
        """One more time step of every site: (trend, new states)."""
        w, p = self.w, self.master
        A = cr.affine(w["W1"], x, p["b1"], "silu")
        if weights8:
            Y, scale, _ = cr.rmsnorm_e4m3(A, p["gamma"])
            (g8, gs), (v8, vs) = weights8["Wg"], weights8["Wv"]
            G = cr.affine(g8, Y, p["bg"], w_scale=gs, x_scale=scale)
            V = cr.affine(v8, Y, p["bv"], "gelu", w_scale=vs, x_scale=scale)
        else:
            Y, _ = cr.rmsnorm(A, p["gamma"])
            G, V = cr.affine(w["Wg"], Y, p["bg"]), cr.affine(w["Wv"], Y, p["bv"], "gelu")
        S, state = cr.gated_step(G, V, state, GATE)
        O = cr.affine(w["Wo"], S, p["bo"], residual=A)   # noqa: E741
        return cr.affine(w["Wh"], O, p["bh"], out_dtype=torch.float32)[0], state


def main(sites=512, observed=384, steps=48, features=16, width=128, rounds=200, rate=0.1, seed=0):
    """Fits the trend at the observed sites, kriges with it, answers one more step; returns what a
    reader or a test looks at."""
    rng = np.random.default_rng(seed)
    n_p = sites - observed
    xy = inputgen.uniform_locations(sites, seed + 1)
    # covariate series: smooth in time, and a truth that is a running mean of one product of them
    x = np.cumsum(rng.normal(size=(sites, steps + 1, features)), axis=1)
    x = (x - x.mean(axis=1, keepdims=True)) / np.sqrt(steps)
    drive = np.tanh(x[:, :, 0] - x[:, :, 1])
    truth = np.zeros(sites)
    for t in range(steps):
        truth = 0.9 * truth + 0.3 * drive[:, t]
    y = truth + 0.05 * rng.normal(size=sites)

    # prediction sites first, like the rest of the package; one series of `steps` columns per site
    X = columns(x[:, :steps].reshape(sites * steps, features).T)
    offsets = torch.arange(0, sites * steps + 1, steps, dtype=torch.int32, device="cuda")
    last = torch.arange(steps - 1, sites * steps, steps, device="cuda")
    target = torch.from_numpy(y).float().cuda()
    net = RecurrentTrend(features, width, seed)
    losses = []
    for _ in range(rounds):
        m, state, kept = net.forward(X, offsets, last)
        err = m - target
        err[:n_p] = 0.0                          # only observed sites teach
        losses.append(float((err ** 2).sum() / observed))
        net.update(net.gradients(2.0 * err / observed, kept), rate)

    m, state, _ = net.forward(X, offsets, last)
    design = np.column_stack([np.ones(sites), m.double().cpu().numpy(), xy[:, 0]])
    V = cr.TileMat(sites, 128)
    cr.cov_build(V, torch.from_numpy(xy).cuda(), "matern", 0.05, 0.1, 1.0, n_pred=n_p, tau2=0.0025)
    Xd = torch.from_numpy(np.ascontiguousarray(design.T)).cuda().T
    W, zhat, _ = cr.krige(V, Xd[n_p:].T.contiguous().T, Xd[:n_p].T.contiguous().T, torch.from_numpy(y[n_p:]).cuda())
    V.close()

    nxt = columns(x[:, steps].T)
    full, s16 = net.step(nxt, state)
    eight, s8 = net.step(nxt, state, net.eight_bits())
    kriged = zhat.cpu().numpy()
    return {"losses": losses, "design": design, "weights": W.cpu().numpy(), "n_pred": n_p,
            "rmse_trend": float(np.sqrt(np.mean((design[:n_p, 1] - truth[:n_p]) ** 2))),
            "rmse_kriged": float(np.sqrt(np.mean((kriged - truth[:n_p]) ** 2))),
            "rmse_mean": float(np.sqrt(np.mean((truth[:n_p] - y[n_p:].mean()) ** 2))),
            "next": full.cpu().numpy(), "next8": eight.cpu().numpy(), "state": s16.cpu().numpy(), "state8": s8.cpu().numpy()}


if __name__ == "__main__":
    r = main()
    print(f"squared error at the observed sites: {r['losses'][0]:.4f} at first, {r['losses'][-1]:.4f} after {len(r['losses'])} rounds")
    print(f"root-mean-square error at the {r['n_pred']} prediction sites: mean {r['rmse_mean']:.3f}, learned trend "
          f"{r['rmse_trend']:.3f}, kriged with it {r['rmse_kriged']:.3f}")
    gap = np.sqrt(np.mean((r["next"] - r["next8"]) ** 2) / np.mean(r["next"] ** 2))
    print(f"next step: 8-bit answers differ from 16-bit ones by {100 * gap:.1f} %")
