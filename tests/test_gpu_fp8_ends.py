"""Products of matrices in 8-bit floating point whose scales lie at the ends of
their range, against the fp64 oracle: a scale is 2^-127 to 2^127, or NaN, for
every product, whatever a single operand's value would be in another format.

The values themselves may leave fp32's range here; the products and their sums
do not, and the bounds are those of tests/fp8_common.py."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import fp8, linear
from oracle.muon import bf16_bits_to_f64, f64_to_bf16_bits
from fp8_common import DEV, cut, device, forward_bounds, host, packed_values
from linear_common import TINY, U, gamma, group_offsets, rounded

pytestmark = pytest.mark.gpu

# Exponents of runs of the contraction, one operand's up and the other's down:
# ordinary, far, and past what bf16 holds of a code (values from 2^-126 to
# 2^128 for every exponent from 17 to 239).
SHIFTS = [0, -120, 60, 110, -110, 115, -115, 119, 0, -104, 120, -60]


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])


def _operand(rows, cols, block, fmt, sign, seed, zeros=()):
    """(codes, exponents, values) whose runs' exponents are 120 + sign SHIFTS, up
    to two more for each row; `zeros`: runs of zeros, at exponent 0 as packed."""
    rng = np.random.default_rng(seed)
    codes, e, _ = packed_values(rng.standard_normal((rows, cols)), block, fmt)
    runs, n = e.shape
    e = np.clip(120 + sign * np.resize(SHIFTS, runs)[:, None] + rng.integers(0, 3, (runs, n)), 0, 254).astype(np.uint8)
    for r in zeros:
        codes[:, 128 * r:128 * r + 128], e[r] = 0, 0
    return codes, e, fp8.unpack(codes, e, block, fmt)


def _weight_gradient(dyt, xt, fmt, wide, accumulate=False, offsets=None, tokens=None, pad=0):
    """fp8_linear_backward's dw of (codes, exponents, values), and its bound."""
    import torch
    ve = _ve()
    N, K, C = dyt[0].shape[0], xt[0].shape[0], xt[0].shape[1]
    T = C if tokens is None else tokens
    E = 1 if offsets is None else len(offsets) - 1
    ref, mag = fp8.weight_gradient(dyt[2], xt[2], offsets, T)
    shape = (N, K + pad) if offsets is None else (E, N, K + pad)
    dw = torch.full(shape, 7.0, dtype=torch.float32 if wide else torch.bfloat16, device=DEV)
    bound = gamma(T + 130) * mag + TINY
    if not wide:
        at = 0
        for e, a, b in linear.parts(offsets, T):
            n = at + -(-(b - a) // 128) * 128
            bound[... if offsets is None else e] += cut(dyt[2][:, at:n], xt[2][:, at:n])
            at = n
    if accumulate:
        held = np.random.default_rng(9).standard_normal((*shape[:-1], K))
        dw[..., :K] = torch.from_numpy(held).to(dw.dtype).to(DEV)
        ref = ref + _host(dw)[..., :K]
        bound = bound + U * (np.abs(ref) + bound)
    off = None if offsets is None else torch.from_numpy(offsets).to(DEV)
    ve.fp8_linear_backward(dy_t=device(*dyt[:2], fmt=fmt), x_t=device(*xt[:2]), dw=dw[..., :K], accumulate=accumulate,
                           offsets=off, tokens=T)
    got = _host(dw)
    assert (got[..., K:] == 7).all()
    return got[..., :K], ref, bound if wide else rounded(bound, ref)


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", fp8.FORMATS)
@pytest.mark.parametrize("N,K,columns,sign,accumulate,pad", [
    (1, 1, 256, 1, False, 0), (64, 72, 1536, 1, False, 0), (130, 257, 1536, -1, True, 3), (264, 136, 640, 1, True, 8),
    (128, 128, 4096, -1, False, 0)])
def test_weight_gradient(N, K, columns, sign, accumulate, pad, fmt, wide):
    print(f"[gpu] fp8 dw at the ends {N}x{K} over {columns} {fmt} fp32 {wide}", flush=True)
    dyt = _operand(N, columns, 1, fmt, sign, 1, zeros=(4,) if columns > 512 else ())
    xt = _operand(K, columns, 1, "e4m3", -sign, 2, zeros=(3,) if columns > 512 else ())
    _within(*_weight_gradient(dyt, xt, fmt, wide, accumulate, pad=pad), "dw")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", fp8.FORMATS)
@pytest.mark.parametrize("low", ["dy", "x"])
def test_weight_gradient_of_the_smallest_codes(low, fmt, wide):
    """Subnormal codes under the smallest exponents, down to 2^-9 2^-127 (E4M3)
    or 2^-16 2^-127 (E5M2), times values that bring them back."""
    rng = np.random.default_rng(10)
    steps = dict(dy=8 if fmt == "e4m3" else 4, x=8)[low]
    q = {}
    for name, rows, f in (("dy", 70, fmt), ("x", 140, "e4m3")):
        codes, e, _ = packed_values(rng.standard_normal((rows, 384)), 1, f)
        if name == low:
            codes = (rng.integers(1, steps, codes.shape) + 128 * rng.integers(0, 2, codes.shape)).astype(np.uint8)
        e = rng.integers(0, 3, e.shape) + (0 if name == low else 248 if f == "e4m3" else 240)
        q[name] = (codes, e.astype(np.uint8), fp8.unpack(codes, e, 1, f))
    _within(*_weight_gradient(q["dy"], q["x"], fmt, wide), "dw")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("groups,tokens", [(5, 900), (70, 2000)])
def test_weight_gradient_of_groups(groups, tokens, wide):
    off = group_offsets(tokens, groups, 3, first=1, spare=2)
    columns = fp8.columns(tokens, groups)
    dyt, xt = _operand(136, columns, 1, "e5m2", 1, 3), _operand(72, columns, 1, "e4m3", -1, 4)
    at = 0
    for _, a, b in linear.parts(off, tokens):   # zeros behind each group's last row, as packed
        n = at + -(-(b - a) // 128) * 128
        for q in (dyt, xt):
            q[0][:, at + b - a:n] = 0
        at = n
    dyt, xt = (*dyt[:2], fp8.unpack(*dyt[:2], 1, "e5m2")), (*xt[:2], fp8.unpack(*xt[:2]))
    _within(*_weight_gradient(dyt, xt, "e5m2", wide, offsets=off, tokens=tokens), "dw")


@pytest.mark.parametrize("path,split", [(2, 0), (2, 1), (3, 1)])
def test_weight_gradient_forms(path, split):
    dyt, xt = _operand(130, 4096, 1, "e4m3", 1, 5), _operand(200, 4096, 1, "e4m3", -1, 6)
    with _ve().options(linear_path=path, linear_split=split):
        for wide in (False, True):
            _within(*_weight_gradient(dyt, xt, "e4m3", wide), "dw")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_weight_gradient_of_packed_bf16(fmt, wide):
    """Packed rows next to the largest bf16 value, which rounds up to a code of
    2^128, times rows next to the smallest ones."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(7)
    T, N, K = 300, 40, 72
    dy = rng.uniform(0.5, 1, (T, N)) * 2.0 ** -124 * rng.choice([-1, 1], (T, N))
    x = rng.uniform(0.99, 0.996, (T, K)) * 2.0 ** 128 * rng.choice([-1, 1], (T, K))
    dy[:, 3], x[:, 5] = dy[:, 3] * 2.0 ** -8, x[:, 5] * 2.0 ** -20
    q = {}
    for name, v, f in (("dy", dy, fmt), ("x", x, "e4m3")):
        bits = f64_to_bf16_bits(v)
        q[name] = ve.new_fp8(v.shape[1], ve.fp8_columns(T), format=f, device=DEV)
        ve.fp8_pack(torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16), None, q[name])
        codes, e = fp8.pack(fp8.transposed(bf16_bits_to_f64(bits).reshape(v.shape))[0], 1, f)
        got, ge = host(q[name])
        assert np.array_equal(got, codes) and np.array_equal(ge, e)
        q[name + "v"] = (codes, e, fp8.unpack(codes, e, 1, f))
    assert np.abs(q["xv"][2]).max() == 2.0 ** 128
    _within(*_weight_gradient(q["dyv"], q["xv"], fmt, wide, tokens=T), "dw")


@pytest.mark.parametrize("wide", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("codes", ["any", "zeros", "positive"])
def test_weight_gradient_of_nan_scales(wide, codes):
    """A NaN scale makes its row or column NaN, whatever the codes, and no other."""
    dyt = _operand(140, 640, 1, "e4m3", 0, 8)
    xt = _operand(130, 640, 1, "e4m3", 0, 9)
    if codes == "zeros":
        dyt[0][7, 128:256] = 0
        xt[0][129, 512:] = 0
    if codes == "positive":
        dyt, xt = (dyt[0] & 127, *dyt[1:]), (xt[0] & 127, *xt[1:])
    dyt[1][1, 7] = xt[1][4, 129] = 255
    dyt, xt = (*dyt[:2], fp8.unpack(*dyt[:2])), (*xt[:2], fp8.unpack(*xt[:2]))
    with np.errstate(invalid="ignore"):
        got, ref, bound = _weight_gradient(dyt, xt, "e4m3", wide)
    nan = np.zeros(got.shape, bool)
    nan[7], nan[:, 129] = True, True
    assert np.array_equal(np.isnan(got), nan)
    fine = np.ix_(np.arange(140) != 7, np.arange(130) != 129)
    _, want, bound = _weight_gradient(tuple(np.delete(v, 7, i) for i, v in zip((0, 1, 0), dyt)),
                                      tuple(np.delete(v, 129, i) for i, v in zip((0, 1, 0), xt)), "e4m3", wide)
    _within(got[fine], want, bound, "dw")


@pytest.mark.parametrize("fmt", fp8.FORMATS)
@pytest.mark.parametrize("T,K,N", [(1, 640, 40), (20, 1536, 72), (130, 640, 200), (300, 1536, 264)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_forward_and_dx(T, K, N, sign, fmt):
    """The same product for a forward pass and for dx, in every form."""
    import torch
    ve = _ve()
    x = _operand(T, K, 1, fmt, sign, 10)
    w = _operand(N, K, 128, "e4m3", -sign, 11)
    ref, z, mag = linear.forward(x[2], w[2])
    bound = forward_bounds(ref, z, mag, cut(x[2], w[2]), K, "none")[1]
    xq, wq = device(*x[:2], fmt=fmt), device(*w[:2], 128)
    for path in (0, 2, 3, 4):
        with ve.options(linear_path=path):
            y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
            ve.fp8_linear_forward(xq, wq, y)
            _within(_host(y), ref, bound, ("y", path))
            ve.fp8_linear_backward(dy=xq, w_t=wq, dx=y.zero_())
            _within(_host(y), ref, bound, ("dx", path))


@pytest.mark.parametrize("sign", [0, 1])
def test_infinities_of_e5m2(sign):
    """An infinity times a value is one, times 0 NaN, and two of opposite sign
    NaN, in every product; elements without one are as ever.  sign 1: beside
    scales at the ends."""
    import torch
    ve = _ve()
    T, K, N = 70, 640, 140
    x, w = _operand(T, K, 1, "e5m2", sign, 12), _operand(N, K, 128, "e4m3", -sign, 13)
    x[0][3, 5], x[0][3, 300], x[0][9, 639], x[0][11, 0], x[0][11, 64] = 0x7C, 0x7C, 0xFC, 0x7C, 0xFC
    w[0][7, 5] = w[0][8, 639] = 0
    x, w = (*x[:2], fp8.unpack(*x[:2], 1, "e5m2")), (*w[:2], fp8.unpack(*w[:2], 128))
    with np.errstate(invalid="ignore"):
        prod = [[x[2][t] * w[2][n] for n in range(N)] for t in (3, 9, 11)]
        want = np.array([[p.sum() for p in row] for row in prod])
    assert np.isinf(want).any() and np.isnan(want).any()
    fine = np.ones(T, bool)
    fine[[3, 9, 11]] = False
    ref, z, mag = linear.forward(x[2][fine], w[2])
    lost = cut(x[2][fine], w[2])
    bound = forward_bounds(ref, z, mag, lost, K, "none")[1]
    exact = gamma(K + 130) * mag + TINY
    xq, wq = device(*x[:2], fmt="e5m2"), device(*w[:2], 128)
    rows = device(w[0], np.repeat(w[1], 128, 1)[:, :N])
    for path in (0, 2, 3, 4):
        with ve.options(linear_path=path):
            out = {k: torch.empty(T, N, dtype=d, device=DEV) for k, d in
                   (("y", torch.bfloat16), ("dx", torch.bfloat16), ("dw", torch.bfloat16), ("dw32", torch.float32))}
            ve.fp8_linear_forward(xq, wq, out["y"])
            ve.fp8_linear_backward(dy=xq, w_t=wq, dx=out["dx"])
            for k in ("dw", "dw32"):
                ve.fp8_linear_backward(dy_t=xq, x_t=rows, dw=out[k], tokens=K)
        for k, t in out.items():
            got = _host(t)
            assert np.array_equal(got[[3, 9, 11]], want, equal_nan=True), (k, path)
            _within(got[fine], ref, exact if k == "dw32" else rounded(exact + lost, ref) if k == "dw" else bound, (k, path))
