"""Definition of the products in 8-bit integers with a scale per token and per
output channel."""
from fractions import Fraction

import numpy as np

from .dense import act as _act

TINY = 2.0 ** -100


def int8_quantize(x):
    """(codes [rows, K], scales float32 [rows]) of the rows of x, whose values are
    float32 numbers: 127 x / max |x| to the nearest whole number, ties to even.
    The float64 quotient decides: it is a tie only where the exact one is, as two
    numbers of 24 bits have quotients at least 2^-32 of a tie apart from it."""
    x = np.asarray(x, dtype=np.float64)
    codes, scales = np.zeros(x.shape, dtype=np.int64), np.zeros(x.shape[0], dtype=np.float32)
    for i, row in enumerate(x):
        top = np.max(np.abs(row))
        if not np.isfinite(row).all():
            scales[i] = np.nan
        elif top >= TINY:
            codes[i] = np.rint(127 * row / top)
            scales[i] = np.float32(top) / np.float32(127)
    return codes, scales


def int8_code_exact(v, top):
    """One code, in exact fractions."""
    q = Fraction(float(v)) * 127 / Fraction(float(top))
    return round(q)          # Python rounds halves to even


def int8_product(x_codes, x_scales, w_codes, w_scales, bias=None, act="none", residual=None):
    """(y, z, the scaled sum): codes [T, K] and [F, K], exact sums in int64."""
    total = np.asarray(x_codes, np.int64) @ np.asarray(w_codes, np.int64).T
    s = total * np.asarray(x_scales, np.float64)[:, None] * np.asarray(w_scales, np.float64)
    z = s if bias is None else s + bias
    y = _act(act, z)[0]
    return (y if residual is None else y + residual), z, s


def int8_experts(x_codes, x_scales, w_codes, w_scales, offsets, bias=None, act="none"):
    """The same for rows sorted by expert: [(first row, last row, y, z, s)] of the experts that have rows."""
    out = []
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a < b:
            out.append((a, b) + int8_product(x_codes[a:b], x_scales[a:b], w_codes[e], w_scales[e],
                                             None if bias is None else bias[e], act))
    return out
