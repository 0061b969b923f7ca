"""Trend-network operators in FP64: the affine product with its epilogue, the root-mean-square
norm, and the gated recurrence, each with its gradient (oracle; test infra).

The paper takes the trend design of universal kriging as given, so these follow the formulas
of include/cr.h alone.  Matrices are features x columns."""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def activation(z: np.ndarray, act: str) -> np.ndarray:
    """act(z): none, relu, silu = z sigmoid(z), gelu = z Phi(z)."""
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    return z


def activation_slope(z: np.ndarray, act: str) -> np.ndarray:
    """act'(z); relu has slope 0 at 0."""
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "silu":
        return _sigmoid(z) * (1.0 + z * _sigmoid(-z))
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def affine(W, X, bias=None, act="none", residual=None, w_scale=None, x_scale=None):
    """(Y, Z): Z = diag(w_scale) W^T X diag(x_scale) + bias 1^T, Y = act(Z) + residual."""
    Z = W.T @ X
    if w_scale is not None:
        Z = Z * w_scale[:, None]
    if x_scale is not None:
        Z = Z * x_scale[None, :]
    if bias is not None:
        Z = Z + bias[:, None]
    Y = activation(Z, act)
    return (Y if residual is None else Y + residual), Z


def affine_backward(W, X, dY, Z, act="none"):
    """(dX, dW, dbias) of sum(dY * affine)."""
    G = dY * activation_slope(Z, act) if act != "none" else dY
    return W @ G, X @ G.T, G.sum(axis=1)


def rmsnorm(X, gamma, residual=None, eps=1e-6):
    """(Y, H): H = X + residual, Y = gamma * H / sqrt(mean(H^2) + eps) by column."""
    H = X if residual is None else X + residual
    return gamma[:, None] * H / np.sqrt(np.mean(H * H, axis=0) + eps), H


def column_scale(Y):
    """The e4m3 scale of each column: max(max|y|, 2^-100) / 448."""
    return np.maximum(np.max(np.abs(Y), axis=0), 2.0 ** -100) / 448.0


def rmsnorm_backward(H, gamma, dY, dH=None, eps=1e-6):
    """(dX, dgamma) of sum(dY * rmsnorm) + sum(dH * H)."""
    r = 1.0 / np.sqrt(np.mean(H * H, axis=0) + eps)
    u = gamma[:, None] * dY
    dX = r * u - H * r ** 3 * np.mean(u * H, axis=0)
    return (dX if dH is None else dX + dH), np.sum(dY * H * r, axis=1)


def gate(g, kind: str):
    """(a, c, da/dg, dc/dg) of h_t = a h_{t-1} + c x_t."""
    if kind == "coeff":
        return g, np.ones_like(g), np.ones_like(g), np.zeros_like(g)
    a, q = _sigmoid(g), _sigmoid(-g)
    if kind == "convex":
        return a, q, a * q, -a * q
    return a, np.sqrt(q * (1.0 + a)), a * q, -a * a * np.sqrt(q / (1.0 + a))


def gated_scan(G, X, kind, offsets, h0):
    """(H, hT) step by step along the packed series."""
    a, c, _, _ = gate(G, kind)
    H, hT = np.empty_like(X), h0.copy()
    for s in range(len(offsets) - 1):
        h = h0[:, s]
        for t in range(offsets[s], offsets[s + 1]):
            h = a[:, t] * h + c[:, t] * X[:, t]
            H[:, t] = h
        hT[:, s] = h
    return H, hT


def gated_scan_backward(G, X, dH, kind, offsets, h0, dhT):
    """(dG, dX, dh0) of sum(dH * H) + sum(dhT * hT)."""
    a, c, da, dc = gate(G, kind)
    H, _ = gated_scan(G, X, kind, offsets, h0)
    dG, dX, dh0 = np.empty_like(X), np.empty_like(X), dhT.copy()
    for s in range(len(offsets) - 1):
        q = dhT[:, s]
        for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
            before = H[:, t - 1] if t > offsets[s] else h0[:, s]
            q = q + dH[:, t]
            dX[:, t] = c[:, t] * q
            dG[:, t] = q * (before * da[:, t] + X[:, t] * dc[:, t])
            q = a[:, t] * q
        dh0[:, s] = q
    return dG, dX, dh0
