"""Plain reference of matrices in 8-bit floating point and of the products on
them, in fp64.

TEST INFRASTRUCTURE.  Only the test suite and the smoke check may use this
module; it shares nothing with the GPU library.

A code's value comes from the format's definition (sign, exponent with bias 7
or 15, mantissa of 3 or 2 bits; E4M3 has one NaN and no infinity, E5M2 has
both).  A block with largest finite magnitude a has the smallest exponent e >=
-127 with a <= MAX 2^e, held as e + 127, and each value v the code nearest to
v 2^-e, ties to even.
"""

from __future__ import annotations

import numpy as np

from . import linear

FORMATS = ("e4m3", "e5m2")
_BITS = {"e4m3": (3, 7), "e5m2": (2, 15)}  # mantissa bits, bias
MAX = {"e4m3": 448.0, "e5m2": 57344.0}


def values(fmt):
    """The value of each of the 256 codes."""
    m, bias = _BITS[fmt]
    c = np.arange(256)
    exp, frac = (c & 127) >> m, c & ((1 << m) - 1)
    v = np.where(exp == 0, frac * 2.0 ** (1 - bias - m), (1 + frac * 2.0 ** -m) * 2.0 ** (exp.astype(float) - bias))
    if fmt == "e4m3":
        v[(c & 127) == 127] = np.nan
    else:
        v[exp == 31] = np.where(frac[exp == 31] == 0, np.inf, np.nan)
    return np.where(c >= 128, -v, v)


def encode(y, fmt):
    """Nearest codes (ties to even) of values of magnitude at most MAX, infinities and NaN."""
    m, bias = _BITS[fmt]
    a = np.abs(np.nan_to_num(np.asarray(y, np.float64), nan=0.0, posinf=0.0, neginf=0.0))
    _, x = np.frexp(a)                                   # a in [2^(x - 1), 2^x)
    x = np.where(a > 0, np.maximum(x - 1, 1 - bias), 1 - bias)
    q = np.rint(a * 2.0 ** (m - x)).astype(np.int64)     # whole steps of the binade, 2^m .. 2^(m + 1)
    # below the smallest normal value the exponent field is 0 and q the mantissa;
    # a q of 2^(m + 1) carries into the next exponent by itself
    code = (x + bias - 1) * (1 << m) + q
    code = np.where(np.isnan(y), 127, code)
    code = np.where(np.isinf(y), 127 if fmt == "e4m3" else 124, code)
    return (code + 128 * np.signbit(y)).astype(np.uint8)


def exponents(amax, fmt):
    """e + 127 of blocks with these largest magnitudes."""
    f, x = np.frexp(np.asarray(amax, np.float64))
    tf, tx = np.frexp(MAX[fmt])
    e = x - tx + (f > tf)
    return np.where(amax > 0, np.maximum(e + 127, 0), 0).astype(np.uint8)


def pack(v, block_rows=1, fmt="e4m3"):
    """(codes [rows, cols], exponents [ceil(cols / 128), ceil(rows / block_rows)])"""
    v = np.asarray(v, np.float64)
    rows, cols = v.shape
    R, C = -(-rows // block_rows), -(-cols // 128)
    p = np.zeros((R * block_rows, C * 128))
    p[:rows, :cols] = v
    b = p.reshape(R, block_rows, C, 128)
    amax = np.where(np.isfinite(b), np.abs(b), 0).max((1, 3))
    e = exponents(amax, fmt)
    codes = encode(b * 2.0 ** (127.0 - e)[:, None, :, None], fmt).reshape(R * block_rows, C * 128)[:rows, :cols]
    return np.ascontiguousarray(codes), np.ascontiguousarray(e.T)


def unpack(codes, e, block_rows=1, fmt="e4m3"):
    rows, cols = codes.shape
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(float) - 127)).T
    return values(fmt)[codes] * np.repeat(np.repeat(s, block_rows, 0)[:rows], 128, 1)[:, :cols]


def columns(rows, groups=1):
    return (rows + 127 * min(groups, rows)) // 128 * 128


def transposed(v, offsets=None):
    """[cols, columns]: the rows of each group as columns, groups in whole runs of 128."""
    rows, cols = v.shape
    out = np.zeros((cols, columns(rows, 1 if offsets is None else len(offsets) - 1)))
    at = 0
    for _, a, b in linear.parts(offsets, rows):
        out[:, at:at + b - a] = v[a:b].T
        at += -(-(b - a) // 128) * 128
    return out, at


def weight_gradient(dy_t, x_t, offsets, tokens):
    """dw (and the sums of absolute products) from transposed values, group by group."""
    E = 1 if offsets is None else len(offsets) - 1
    dw, mag, at = np.zeros((E, dy_t.shape[0], x_t.shape[0])), np.zeros((E, dy_t.shape[0], x_t.shape[0])), 0
    for e, a, b in linear.parts(offsets, tokens):
        n = -(-(b - a) // 128) * 128
        dw[e] = dy_t[:, at:at + n] @ x_t[:, at:at + n].T
        mag[e] = np.abs(dy_t[:, at:at + n]) @ np.abs(x_t[:, at:at + n]).T
        at += n
    return (dw[0], mag[0]) if offsets is None else (dw, mag)
