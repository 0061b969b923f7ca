"""A trend learned over whole fields, trained by orthogonalised updates, as a column of the kriging design.

Every time step is a field of sites with their covariates.  A block that sees the field as a whole gives each site's trend,

    A = W1^T X + b1;  Y = silu(groupnorm(A));  V = silu(W2^T Y) * (W3^T Y);  O = Wd^T V + A;  m = Wh^T O + bh

with the norm's statistics over each field's sites, is fitted to the observed sites of earlier fields and of the last one, and
m at the last field becomes a column of the kriging design next to the constant.  Matrices take steps along their orthogonalised
gradients (with momentum), whose size does not depend on the gradients'; vectors take gradient steps.

    python examples/field_trend.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import inputgen                                # noqa: E402
import mixed_precision_dense_mat_gb300 as cr   # noqa: E402

GROUPS = 8


def columns(a):
    """A (rows, columns) array as a column-major BF16 CUDA matrix."""
    return torch.from_numpy(np.ascontiguousarray(a.T)).cuda().bfloat16().T


class FieldTrend:
    """The block's parameters: FP32 masters, the BF16 weights that the products read, and the matrices' momentum."""

    def __init__(self, features, width, hidden, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(k, n):
            return (torch.randn((n, k), generator=gen, device="cuda") * k ** -0.5).T

        self.master = {"W1": weight(features, width), "W23": weight(width, 2 * hidden), "Wd": weight(hidden, width),
                       "Wh": weight(width, 1), "b1": torch.zeros(width, device="cuda"), "bh": torch.zeros(1, device="cuda"),
                       "gamma": torch.ones(width, device="cuda"), "beta": torch.zeros(width, device="cuda")}
        self.momentum = {n: torch.zeros_like(m) for n, m in self.master.items() if m.dim() == 2}
        self.round()

    def round(self):
        self.w = {n: m.T.contiguous().bfloat16().T for n, m in self.master.items() if m.dim() == 2}

    def update(self, grads, rate, keep=0.9):
        for n, g in grads.items():
            if n in self.momentum:
                m = self.momentum[n].mul_(keep).add_(g)
                k, c = m.shape
                # singular values near 1 spread over an entry's share of them
                self.master[n] -= rate * (max(k, c) ** -0.5) * cr.orthogonalize(m, out_dtype=torch.bfloat16).float()
            else:
                self.master[n] -= rate * g / (1.0 + g.norm())
        self.round()

    def forward(self, X, offsets):
        w, p = self.w, self.master
        A = cr.affine(w["W1"], X, p["b1"])
        Y, mean, rstd = cr.group_norm(A, GROUPS, p["gamma"], p["beta"], "silu", offsets, save=True)
        V, Z = cr.gated_affine(w["W23"], Y, act="silu", save=True)
        O = cr.affine(w["Wd"], V, residual=A)   # noqa: E741
        m = cr.affine(w["Wh"], O, p["bh"], out_dtype=torch.float32)[0]
        return m, (X, offsets, A, Y, mean, rstd, V, Z, O)

    def gradients(self, dm, kept):
        X, offsets, A, Y, mean, rstd, V, Z, O = kept   # noqa: E741
        w, p, f32 = self.w, self.master, torch.float32
        dO, dWh, dbh = cr.affine_backward(w["Wh"], O, dm[None].bfloat16(), dw_dtype=f32)
        dV, dWd, _ = cr.affine_backward(w["Wd"], V, dO, need=(True, True, False), dw_dtype=f32)
        dY, dW23, _ = cr.gated_affine_backward(w["W23"], Y, dV, Z, "silu", need=(True, True, False), dw_dtype=f32)
        dA, dgamma, dbeta = cr.group_norm_backward(A, GROUPS, p["gamma"], p["beta"], dY, mean, rstd, "silu", offsets)
        _, dW1, db1 = cr.affine_backward(w["W1"], X, dA + dO, need=(False, True, True), dw_dtype=f32)
        return {"W1": dW1, "W23": dW23, "Wd": dWd, "Wh": dWh, "b1": db1, "bh": dbh, "gamma": dgamma, "beta": dbeta}


def main(sites=512, observed=384, fields=24, features=16, width=64, hidden=128, rounds=120, rate=0.03, seed=0):
    """Fits the trend at the observed sites of all fields, kriges the last field with it; returns what a reader or a test looks at."""
    rng = np.random.default_rng(seed)
    n_p = sites - observed
    xy = inputgen.uniform_locations(sites, seed + 1)
    # covariates of every field, on a level and a scale of its own; a truth that looks at them relative to the field
    x = rng.normal(size=(fields, sites, features)) * rng.uniform(0.5, 2.0, (fields, 1, 1)) + rng.normal(size=(fields, 1, 1))
    rel = (x - x.mean(axis=(1, 2), keepdims=True)) / x.std(axis=(1, 2), keepdims=True)
    truth = np.tanh(rel[:, :, 0]) * rel[:, :, 1] + 0.5 * rel[:, :, 2]
    y = truth + 0.05 * rng.normal(size=truth.shape)

    # prediction sites first, like the rest of the package; one field after the other
    X = columns(x.reshape(fields * sites, features).T)
    offsets = torch.arange(0, fields * sites + 1, sites, dtype=torch.int32, device="cuda")
    target = torch.from_numpy(y.reshape(-1)).float().cuda()
    taught = (torch.arange(fields * sites, device="cuda") % sites) >= n_p
    net = FieldTrend(features, width, hidden, seed)
    losses = []
    for _ in range(rounds):
        m, kept = net.forward(X, offsets)
        err = torch.where(taught, m - target, torch.zeros_like(m))
        losses.append(float((err ** 2).sum() / taught.sum()))
        net.update(net.gradients(2.0 * err / taught.sum(), kept), rate)

    m, _ = net.forward(X, offsets)
    trend = m[-sites:].double().cpu().numpy()
    design = np.column_stack([np.ones(sites), trend, xy[:, 0]])
    V = cr.TileMat(sites, 128)
    cr.cov_build(V, torch.from_numpy(xy).cuda(), "matern", 0.05, 0.1, 1.0, n_pred=n_p, tau2=0.0025)
    Xd = torch.from_numpy(np.ascontiguousarray(design.T)).cuda().T
    _, zhat, _ = cr.krige(V, Xd[n_p:].T.contiguous().T, Xd[:n_p].T.contiguous().T, torch.from_numpy(y[-1, n_p:].copy()).cuda())
    V.close()
    kriged = zhat.cpu().numpy()
    return {"losses": losses, "design": design, "n_pred": n_p, "kriged": kriged,
            "rmse_trend": float(np.sqrt(np.mean((trend[:n_p] - truth[-1, :n_p]) ** 2))),
            "rmse_kriged": float(np.sqrt(np.mean((kriged - truth[-1, :n_p]) ** 2))),
            "rmse_mean": float(np.sqrt(np.mean((truth[-1, :n_p] - y[-1, n_p:].mean()) ** 2)))}


if __name__ == "__main__":
    r = main()
    print(f"squared error at the observed sites: {r['losses'][0]:.4f} at first, {r['losses'][-1]:.4f} after {len(r['losses'])} rounds")
    print(f"root-mean-square error at the {r['n_pred']} prediction sites of the last field: mean {r['rmse_mean']:.3f}, learned trend "
          f"{r['rmse_trend']:.3f}, kriged with it {r['rmse_kriged']:.3f}")
