"""fp64 CPU oracle of the 8-bit activation checkpoints: the codes and scales of a saved
activation, the values they stand for, and the activation and its gradient from them.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.

Blocks of 32 consecutive features of a segment (all F for GELU, each shard's gate and each
shard's up features for SwiGLU) share a power-of-two scale 2^k, k the largest integer <= 126
with amax 2^k <= 127 (0 for zeros); a code is rint(z 2^k), ties to even; the scale byte is
127 - k, or 255 for a block with a non-finite value, which stands for NaN.  A block whose amax is
bf16's largest value has k = -121 (at -122 its code would stand for 2^128) and rounds ties towards
zero.
"""
from __future__ import annotations

import numpy as np

from .mlp import silu, silu_grad

BLOCK = 32
LARGEST = 255.0 * 2.0 ** 120  # of bf16


def segments(ffn, tp, act):
    """(segments of a row of Z, features of each)."""
    return (2 * tp, ffn // tp) if act == "swiglu" else (1, ffn)


def quantize(Z, ffn, tp, act):
    """(codes int8 [T][F1], scale bytes uint8 [T][blocks])."""
    n, width = segments(ffn, tp, act)
    T = Z.shape[0]
    z = np.asarray(Z, dtype=np.float64).reshape(T, n, width)
    nb = -(-width // BLOCK)
    codes = np.zeros((T, n, width), np.int8)
    scales = np.zeros((T, n, nb), np.uint8)
    for t in range(T):
        for s in range(n):
            for b in range(nb):
                blk = z[t, s, b * BLOCK:(b + 1) * BLOCK]
                if not np.isfinite(blk).all():
                    scales[t, s, b] = 255
                    continue
                amax = np.abs(blk).max()
                k = 0
                if amax > 0:
                    k = 300
                    while amax * 2.0 ** k > 127.0:
                        k -= 1
                    k = max(-121, min(k, 126))
                scales[t, s, b] = 127 - k
                q = blk * 2.0 ** k
                if amax == LARGEST:
                    q = q * (1.0 - 2.0 ** -24)
                codes[t, s, b * BLOCK:(b + 1) * BLOCK] = np.rint(q)
    return codes.reshape(T, n * width), scales.reshape(T, n * nb)


def decode(codes, scales, ffn, tp, act):
    """The float64 values [T][F1] that the codes stand for."""
    n, width = segments(ffn, tp, act)
    T = codes.shape[0]
    nb = -(-width // BLOCK)
    step = np.ldexp(1.0, scales.astype(np.int64) - 127)
    step = np.where(scales == 255, np.nan, step).reshape(T, n, nb)
    per = np.repeat(step, BLOCK, axis=2)[:, :, :width]
    return (codes.astype(np.float64).reshape(T, n, width) * per).reshape(T, n * width)


def _sigmoid(x):
    """1 / (1 + e^-x) without overflow; exact relative to its value for x << 0."""
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


_K, _C = np.sqrt(2.0 / np.pi), 0.044715


def gelu(z):
    """The tanh form as z sigmoid(2u): 0.5 z (1 + tanh(u)) itself loses its value for z << 0,
    where 1 + tanh(u) cancels (2^-53 of 1 against e^2u)."""
    return z * _sigmoid(2.0 * _K * (z + _C * z ** 3))


def gelu_grad(z):
    s = _sigmoid(2.0 * _K * (z + _C * z ** 3))
    r = _sigmoid(-2.0 * _K * (z + _C * z ** 3))  # 1 - s
    return s + z * s * r * 2.0 * _K * (1.0 + 3.0 * _C * z * z)


def _gate_up(z, ffn, tp):
    v = z.reshape(z.shape[0], tp, 2, ffn // tp)
    return v[:, :, 0], v[:, :, 1]


def act(z, ffn, tp, kind):
    if kind == "gelu":
        return gelu(z)
    g, u = _gate_up(z, ffn, tp)
    return (silu(g) * u).reshape(z.shape[0], ffn)


def act_grad(dA, z, ffn, tp, kind):
    if kind == "gelu":
        return dA * gelu_grad(z)
    g, u = _gate_up(z, ffn, tp)
    d = dA.reshape(g.shape)
    return np.stack([d * u * silu_grad(g), d * silu(g)], axis=2).reshape(z.shape)
