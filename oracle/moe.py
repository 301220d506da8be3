"""fp64 CPU oracle of the mixture-of-experts MLP for a few tokens.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.

    l = X Wr^T;  ids = the topk largest l (equal ones by index);  w = softmax(l)[ids]
    Y_t = sum over t's experts of w W2_e act(W1_e x_t)
"""
from __future__ import annotations

import numpy as np

from .act8 import _sigmoid, gelu


def route(X, Wr, topk, normalize):
    """(logits [T][E], ids [T][topk], weights [T][topk])."""
    l = X @ Wr.T
    ids = np.argsort(-l, axis=1, kind="stable")[:, :topk]
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, ids, 1)
    if normalize:
        w = w / w.sum(1, keepdims=True)
    return l, ids, w


def activation(x, W1e, kind):
    """(a, z): act of one expert's fc1 for one token, and the pre-activations."""
    if kind == "gelu":
        z = W1e @ x
        return gelu(z), z
    g, u = W1e[0] @ x, W1e[1] @ x
    return g * _sigmoid(g) * u, np.stack([g, u])


def forward(X, W1, W2, ids, w, kind):
    """Y for a given routing."""
    Y = np.zeros((X.shape[0], W2.shape[1]))
    for t in range(X.shape[0]):
        for k, e in enumerate(ids[t]):
            Y[t] += w[t, k] * (W2[e] @ activation(X[t], W1[e], kind)[0])
    return Y
