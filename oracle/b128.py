"""fp64 CPU oracle of block-scaled E4M3: the codes' values and scale exponents of a matrix, and
the three products of a linear layer on them.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module.

Blocks of 128 consecutive columns of a row, or of 128 x 128, share a scale 2^-k, k the largest
integer <= 126 with amax 2^k <= 448 (0 for zeros); a block with a non-finite value stands for NaN.
E4M3 values are found in the sorted list of all of them, ties to the even code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values():
    """The 127 non-negative finite values by code: 2^(e - 7) (1 + m / 8), subnormals m 2^-9."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, 2.0 ** (e - 7.0) * (1 + m / 8))


_VALUES = e4m3_values()


def round_e4m3(x):
    """x (|x| <= 448) to the nearest E4M3 value, ties to the even code."""
    a = np.abs(x)
    hi = np.minimum(np.searchsorted(_VALUES, a), 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - _VALUES[lo], _VALUES[hi] - a
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return np.copysign(np.where(up, _VALUES[hi], _VALUES[lo]), x)


def scale_exponent(amax):
    """k of a block with this finite largest magnitude."""
    amax = float(amax)
    if amax == 0:
        return 0
    k = 126
    while amax > 448 * 2.0 ** -k:
        k -= 1
    return k


def quantize(x, square=False):
    """(values [R][C] that the codes stand for, scale bytes [row blocks][column blocks])."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    rows = BLOCK if square else 1
    out = np.empty_like(x)
    scales = np.empty((-(-R // rows), -(-C // BLOCK)), np.int64)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * rows, (i + 1) * rows), slice(j * BLOCK, (j + 1) * BLOCK))
            b = x[at]
            if not np.isfinite(b).all():
                out[at], scales[i, j] = np.nan, 255
                continue
            k = scale_exponent(np.abs(b).max())
            out[at], scales[i, j] = round_e4m3(b * 2.0 ** k) * 2.0 ** -k, 127 - k
    return out, scales


def linear(X, W, dY=None):
    """(Y, dX, dW, and of each the sum of the products' magnitudes) of the layer y = x W^T."""
    xq, wq = quantize(X)[0], quantize(W, True)[0]
    out = dict(Y=(xq @ wq.T, np.abs(xq) @ np.abs(wq).T))
    if dY is not None:
        d, dt, xt = quantize(dY)[0], quantize(np.asarray(dY).T)[0], quantize(np.asarray(X).T)[0]
        out["dX"] = (d @ wq, np.abs(d) @ np.abs(wq))
        out["dW"] = (dt @ xt.T, np.abs(dt) @ np.abs(xt).T)
    return out
