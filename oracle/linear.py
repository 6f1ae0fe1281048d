"""Plain reference of the linear layer's operators and of 8-bit saved
activations, in fp64.

TEST INFRASTRUCTURE.  Only the test suite and the smoke check may use this
module; it shares nothing with the GPU library.

Everything is evaluated from the formulas in fp64 without intermediate
rounding, group by group:

    z = x w^T + bias, y = act(z) + residual
    dz = dy act'(z), dx = dz w + dx_add, dw = dz^T x, dbias = sum dz

A saved activation is (codes, scales) by the code's rule in fp32 arithmetic,
operation by operation, so that the GPU's codes can be compared bit for bit.
"""

from __future__ import annotations

import numpy as np
from scipy.special import erfc

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_C = np.sqrt(2.0 / np.pi)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def act(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.where(z <= 0, 0.0, z)
    if name == "none":
        return z.copy()
    with np.errstate(all="ignore"):
        if name == "gelu":
            y = z * 0.5 * erfc(-z / np.sqrt(2.0))
        elif name == "gelu_tanh":
            y = z * _sigmoid(2 * _C * (z + 0.044715 * z ** 3))
        else:
            y = z * _sigmoid(z)
    return np.where(z == -np.inf, 0.0, y)


def slope(name, z):
    z = np.asarray(z, np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    with np.errstate(all="ignore"):
        if name == "gelu":
            d = 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        elif name == "gelu_tanh":
            u = 2 * _C * (z + 0.044715 * z ** 3)
            q, e = _sigmoid(u), np.exp(-np.abs(u))
            d = q + z * e / (1 + e) ** 2 * 2 * _C * (1 + 3 * 0.044715 * z * z)
        else:
            q, e = _sigmoid(z), np.exp(-np.abs(z))
            d = q + z * e / (1 + e) ** 2
    d = np.where(z == np.inf, 1.0, d)
    return np.where(z == -np.inf, 0.0, d)


def parts(offsets, tokens):
    if offsets is None:
        return [(0, 0, tokens)]
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(offsets[:-1], offsets[1:]))]


def forward(x, w, bias=None, name="none", residual=None, offsets=None):
    """(y, z, mag): mag = the sums of absolute products (for error bounds);
    rows of no group are NaN."""
    T, N = x.shape[0], w.shape[-2]
    z = np.full((T, N), np.nan)
    mag = np.zeros((T, N))
    for e, a, b in parts(offsets, T):
        we = w if offsets is None else w[e]
        z[a:b] = x[a:b] @ we.T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(we).T
        if bias is not None:
            be = bias if offsets is None else bias[e]
            z[a:b] += be
            mag[a:b] += np.abs(be)
    y = act(name, z)
    if residual is not None:
        y = y + residual
    return y, z, mag


def backward(dy, w, x=None, z=None, name="none", dx_add=None, offsets=None):
    """dict of dx, dw, dbias, dz (rows of no group: NaN in dx and dz)."""
    T, N = dy.shape
    K = w.shape[-1]
    E = 1 if offsets is None else len(offsets) - 1
    dz = dy * (slope(name, z) if name != "none" else 1.0)
    dx, dw, db = np.full((T, K), np.nan), np.zeros((E, N, K)), np.zeros((E, N))
    for e, a, b in parts(offsets, T):
        dx[a:b] = dz[a:b] @ (w if offsets is None else w[e])
        if x is not None:
            dw[e] = dz[a:b].T @ x[a:b]
        db[e] = dz[a:b].sum(0)
    if dx_add is not None:
        dx = dx + dx_add
    if offsets is None:
        dw, db = dw[0], db[0]
    return dict(dx=dx, dw=dw, dbias=db, dz=dz)


def pack(v, block):
    """fp32 matrix -> (codes int8, scales fp32), each operation in fp32."""
    v = np.ascontiguousarray(v, np.float32)
    rows, cols = v.shape
    runs = -(-cols // block)
    pad = np.zeros((rows, runs * block), np.float32)
    pad[:, :cols] = v
    r = pad.reshape(rows, runs, block)
    with np.errstate(all="ignore"):
        amax = np.abs(r).max(-1, keepdims=True)
        bad = ~np.isfinite(amax)
        up = np.where(amax < np.float32(2.0 ** -100), np.float32(2.0 ** 64), np.float32(1))
        inv = np.where(amax > 0, np.float32(127) / (amax * up), np.float32(0)).astype(np.float32)
        q = np.rint((r * up).astype(np.float32) * inv)
        q = np.where(bad | (amax == 0), 0, np.clip(q, -127, 127))
        scale = np.where(bad, np.float32(np.nan), (amax / np.float32(127)).astype(np.float32))
    codes = np.nan_to_num(q).astype(np.int8).reshape(rows, -1)[:, :cols]
    return np.ascontiguousarray(codes), np.ascontiguousarray(scale[..., 0].astype(np.float32))


def unpack(codes, scales, block):
    """fp32 products code * scale (before the rounding to bf16)."""
    wide = np.repeat(scales, block, axis=1)[:, :codes.shape[1]]
    with np.errstate(all="ignore"):
        return codes.astype(np.float32) * wide
