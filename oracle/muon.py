"""fp64 CPU oracle of the orthogonalised update: Newton-Schulz steps on a normalised matrix, the
momentum and the weight's update; and the same steps with the library's operands rounded to fp16,
which says how far those roundings move a given input's result.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.
"""
from __future__ import annotations

import numpy as np

COEF = (3.4445, -4.7750, 2.0315)


def normalized(U):
    U = np.asarray(U, np.float64)
    n = np.linalg.norm(U)
    return U / n if n else U


def orthogonalize(U, steps=5, coef=COEF):
    """By singular values: U = P S Q^T goes to P p(...p(S / |U|)) Q^T."""
    a, b, c = coef
    X = normalized(U)
    P, s, Q = np.linalg.svd(X, full_matrices=False)
    for _ in range(steps):
        s = s * (a + b * s ** 2 + c * s ** 4)
    return (P * s) @ Q


def by_products(U, steps=5, coef=COEF):
    a, b, c = coef
    X = normalized(U)
    for _ in range(steps):
        if X.shape[0] <= X.shape[1]:
            A = X @ X.T
            X = a * X + (b * A + c * A @ A) @ X
        else:
            A = X.T @ X
            X = a * X + X @ (b * A + c * A @ A)
    return X


def _half(x, scale):
    return (x * scale).astype(np.float16).astype(np.float64) / scale


def rounded(U, steps=5, coef=COEF):
    """With X, the part of A off its diagonal and that of b A + c A A + a I as fp16 operands, scaled
    by 2^12, 2^12 and 2^10, diagonals apart, and X in two fp16 parts between the steps (one before
    the last), the low one of which goes with the diagonal beta in the last steps and with a before."""
    a, b, c = coef
    X = normalized(U)
    tall = X.shape[0] > X.shape[1]
    if tall:
        X = X.T
    for i in range(steps):
        hi = _half(X, 4096.0)
        lo = _half(X - hi, 4096.0) if i < steps - 1 else 0.0
        A = hi @ hi.T
        d = np.diag(A).copy()
        E = _half(A - np.diag(d), 4096.0)
        EE = E @ E
        beta = a + b * d + c * d * d + c * np.diag(EE)
        D = (b + c * (d[:, None] + d)) * E + c * EE
        D = _half(D - np.diag(np.diag(D)), 1024.0)
        low = beta[:, None] if i >= steps - 3 else a
        X = beta[:, None] * hi + low * lo + D @ hi
    return X.T if tall else X


def step(W, M, G, lr, momentum, nesterov, decay, scale, steps=5, coef=COEF):
    """(W, M, O) after one step on one matrix, and the update U."""
    M = momentum * np.asarray(M, np.float64) + G
    U = G + momentum * M if nesterov else M
    O = orthogonalize(U, steps, coef)
    return (1 - lr * decay) * np.asarray(W, np.float64) - lr * scale * O, M, O, U
