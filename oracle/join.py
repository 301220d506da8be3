"""fp64 CPU oracle of the join between two blocks: norms, gate and residual scale, forward and
backward.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.

    P = norm_post(Y);  h = alpha X + gate[group] P;  Xn = norm_pre(store(h))

``store`` rounds the stream as it is kept (bf16 streams); the pre-norm is that of the stored
value, and the backward takes the stored stream as given.
"""
from __future__ import annotations

import numpy as np


def norm(x, kind, eps):
    """(xhat, mean, 1/sqrt(...)) of each row."""
    if kind == "none":
        z = np.zeros((x.shape[0], 1))
        return x, z, z
    mu = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((x.shape[0], 1))
    rs = 1.0 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    return (x - mu) * rs, mu, rs


def _affine(xh, kind, gamma, beta):
    if kind == "none":
        return xh
    return xh * gamma + (beta if kind == "layer" else 0.0)


def gate_rows(gate, T):
    """The gate of each row: [T][H] (ones without a gate)."""
    if gate is None:
        return 1.0
    return np.repeat(gate, T // gate.shape[0], axis=0)


def forward(X, Y, alpha, gate, post, gamma_post, beta_post, pre, gamma_pre, beta_pre, eps,
            store=lambda h: h):
    T = X.shape[0]
    yh, my, ry = norm(Y, post, eps)
    P = _affine(yh, post, gamma_post, beta_post)
    h = store(alpha * X + gate_rows(gate, T) * P)
    hh, mh, rh = norm(h, pre, eps)
    Xn = _affine(hh, pre, gamma_pre, beta_pre) if pre != "none" else None
    return dict(Xout=h, Xn=Xn, stats=np.concatenate([my, ry, mh, rh], 1))


def norm_grad(u, xh, rs, kind):
    """Gradient through xh = (x - mu) rs for a gradient u of xh."""
    if kind == "none":
        return u
    d = u - xh * (u * xh).mean(1, keepdims=True)
    if kind == "layer":
        d = d - u.mean(1, keepdims=True)
    return rs * d


def backward(X, Y, Xout, alpha, gate, post, gamma_post, beta_post, pre, gamma_pre, eps, dXout,
             dXn):
    """Statistics are those of the given Y and Xout."""
    T, H = X.shape
    out = {}
    dh = np.zeros((T, H)) if dXout is None else dXout
    if pre != "none":
        hh, _, rh = norm(Xout, pre, eps)
        dh = dh + norm_grad(dXn * gamma_pre, hh, rh, pre)
        out["dgamma_pre"] = (dXn * hh).sum(0)
        if pre == "layer":
            out["dbeta_pre"] = dXn.sum(0)
    out["dX"] = alpha * dh
    out["dres_scale"] = np.array([(dh * X).sum()])
    yh, _, ry = norm(Y, post, eps)
    P = _affine(yh, post, gamma_post, beta_post)
    dP = gate_rows(gate, T) * dh
    if gate is not None:
        out["dgate"] = (dh * P).reshape(gate.shape[0], -1, H).sum(1)
    if post != "none":
        out["dgamma_post"] = (dP * yh).sum(0)
        if post == "layer":
            out["dbeta_post"] = dP.sum(0)
        dP = norm_grad(dP * gamma_post, yh, ry, post)
    out["dY"] = dP
    return out
