"""The int8 linear layer, its 8-bit rows and its backward: the oracle.

TEST INFRASTRUCTURE ONLY (same rule as ``oracle.attention``).

Row m of a matrix becomes codes c = rint(127 x / absmax), half to even, of the exact quotient
(integer arithmetic below, no floating division), and a scale s = fp32(absmax / 127); a zero row
has c = 0, s = 1, a row with an infinity or NaN c = 0, s = NaN.
    y = s_x s_w (c_x . c_w) + bias,   dW = dY^T (s_x c_x),   dX = dY (s_w c_w)
"""
from __future__ import annotations

import numpy as np


def quant_rows(x):
    """x: fp32 array of values with at most 24 significant bits -> (int8 codes, fp32 scales)."""
    x = np.asarray(x, np.float32)
    codes, scales = np.zeros(x.shape, np.int8), np.ones(x.shape[0], np.float32)
    for m, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[m] = np.nan
            continue
        top = np.abs(row).max(initial=np.float32(0))
        if top == 0:
            continue
        scales[m] = np.float32(top) / np.float32(127)
        # every value as an integer multiple of 2^-149 (fp32's smallest), exactly
        mant, exp = np.frexp(row.astype(np.float64))
        whole = [int(a * 2 ** 53) << (int(e) - 53 + 149 + 53) for a, e in zip(mant, exp)]
        t = max(abs(a) for a in whole)
        for k, a in enumerate(whole):
            lo, rest = divmod(127 * abs(a), t)
            up = 2 * rest > t or (2 * rest == t and lo % 2 == 1)
            codes[m, k] = (lo + up) * (1 if a >= 0 else -1)
    return codes, scales


def values(codes, scales):
    """The values that 8-bit rows stand for, fp64."""
    return codes.astype(np.float64) * scales.astype(np.float64)[:, None]


def linear(codes, scales, w_codes, w_scales, bias=None):
    """(y, |y| terms' magnitude before the bias is added) in fp64 from the codes."""
    acc = codes.astype(np.int64) @ w_codes.astype(np.int64).T
    y0 = acc * scales.astype(np.float64)[:, None] * w_scales.astype(np.float64)[None, :]
    return (y0 if bias is None else y0 + bias), np.abs(y0)


def grad_weight(dy, codes, scales):
    """(dW, its terms' magnitudes summed) in fp64."""
    x = values(codes, scales)
    return dy.T @ x, np.abs(dy).T @ np.abs(x)


def grad_input(dy, w_codes, w_scales):
    """(dX, its terms' magnitudes summed) in fp64."""
    w = values(w_codes, w_scales)
    return dy @ w, np.abs(dy) @ np.abs(w)
