"""Error bounds of the linear layer's GPU results against the fp64 oracle.

u = 2^-23 covers one fp32 rounding or truncation.  A product over K terms is
within gamma(K) sum |a b| of the exact one (products of bf16 are exact in
fp32).  The activations and slopes are evaluated in fp32 from approximations
whose absolute error is at most A = 2^-18 of max(|z|, 1) (tail fit 1.6e-6
relative of a tail of at most 1/2; exp2 of an argument a with relative error
u has relative error a ln2 u, which times e^-a is below u; reciprocal and the
remaining steps a few u; the product with z or with z du, at most 10 where
the exponential has not vanished, brings the factor): 2^-18 = 3.8e-6 holds
both.  Their slopes are at most 1.2 and the second derivatives at most 1, which carries the error
of z into act(z).  Rounding to bf16 is off by at most 2^-8 of the value.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -23
A = 2.0 ** -18
BF16 = 2.0 ** -8
TINY = 2.0 ** -126


def gamma(k):
    return k * U / (1 - k * U)


def rounded(err, ref):
    """Bound after rounding to bf16 a value within err of ref."""
    return err + BF16 * (np.abs(ref) + err) + TINY


def forward_bounds(ref_y, z, mag, K, name, residual=None):
    """(bound of the fp32 z, bound of the stored y)"""
    ez = gamma(K + 2) * mag + TINY
    ey = ez if name == "none" else 1.2 * ez + A * np.maximum(np.abs(z), 1.0) * (0 if name == "relu" else 1)
    if residual is not None:
        ey = ey + U * (np.abs(ref_y) + ey)
    return ez, rounded(ey, ref_y)


def backward_bounds(ref, dy, w, x, name, offsets, grad_fp32, dx_add=None, before=None):
    """dict of elementwise bounds of dx, dw, dbias.  before: what dw and
    dbias held (accumulate), as (dw, dbias)."""
    from oracle import linear
    dz = np.abs(ref["dz"])
    # fp32 evaluation of dz, then (with an activation) its rounding to bf16
    e32 = U * dz + (0 if name in ("none", "relu") else 2 * A) * np.abs(dy)
    eb = e32 if name == "none" else rounded(e32, dz)
    T, N = dy.shape
    K = w.shape[-1]
    bdx = np.zeros((T, K))
    E = 1 if offsets is None else len(offsets) - 1
    bdw, bdb = np.zeros((E, N, K)), np.zeros((E, N))
    for e, a, b in linear.parts(offsets, T):
        we = np.abs(w if offsets is None else w[e])
        bdx[a:b] = eb[a:b] @ we + gamma(N + 2) * ((dz[a:b] + eb[a:b]) @ we)
        if x is not None:
            ax = np.abs(x[a:b])
            bdw[e] = eb[a:b].T @ ax + gamma(b - a + 34) * ((dz[a:b] + eb[a:b]).T @ ax)
        bdb[e] = e32[a:b].sum(0) + gamma(b - a + 8) * (dz[a:b] + e32[a:b]).sum(0)
    if offsets is None:
        bdw, bdb = bdw[0], bdb[0]
    if dx_add is not None:
        bdx = bdx + U * (np.abs(ref["dx"]) + bdx)
    out = dict(dx=rounded(bdx, ref["dx"]))
    for key, bound, held in (("dw", bdw, None if before is None else before[0]),
                             ("dbias", bdb, None if before is None else before[1])):
        r = ref[key] if held is None else ref[key] + held
        if held is not None:
            bound = bound + U * (np.abs(r) + bound)
        out[key] = bound + TINY if grad_fp32 else rounded(bound, r)
    return out


def group_offsets(tokens, groups, seed, first=0, spare=0):
    """Ragged offsets: `first` rows before the first group and `spare` behind
    the last, about one group in five empty."""
    rng = np.random.default_rng(seed)
    inner = tokens - first - spare
    share = rng.exponential(size=groups) * (rng.random(groups) > 0.2)
    if share.sum() == 0:
        share[-1] = 1
    at = np.rint(np.concatenate([[0], np.cumsum(share)]) / share.sum() * inner).astype(np.int64)
    return first + at
