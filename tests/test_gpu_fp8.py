"""GPU results on matrices in 8-bit floating point against the fp64 oracle
(oracle/fp8.py): packing bit for bit, products within the elementwise bounds of
tests/fp8_common.py."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import fp8, linear
from oracle.muon import bf16_bits_to_f64, f64_to_bf16_bits
from fp8_common import DEV, cut, cut_rows, device, forward_bounds, host, packed_values
from linear_common import A, BF16, TINY, U, gamma, group_offsets, rounded

pytestmark = pytest.mark.gpu


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _bits(shape, seed, spread=0.0):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape)
    return f64_to_bf16_bits(v * np.exp(spread * rng.standard_normal(shape)) if spread else v)


def _up(bits):
    return bf16_bits_to_f64(bits).reshape(bits.shape)


def _dev(bits, pad=0, shift=0):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    rows, cols = t.numel() // t.shape[-1], t.shape[-1]
    flat = torch.full((shift + rows * (cols + pad) + 64,), 0x7FC0, dtype=torch.int16)
    flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = t.reshape(rows, cols)
    strides = [cols + pad, 1] if t.dim() == 2 else [t.shape[1] * (cols + pad), cols + pad, 1]
    return torch.as_strided(flat.to(DEV), t.shape, strides if t.dim() > 1 else [1], shift).view(torch.bfloat16)


def _filled(rows, cols, block=1, fmt="e4m3", groups=None):
    """An Fp8 whose every byte is a marker."""
    q = _ve().new_fp8(rows, cols, block, fmt, groups, DEV)
    import torch
    for t in (q.codes.view(torch.uint8), q.scales):
        base = torch.as_strided(t, (t.untyped_storage().nbytes(),), (1,), 0)
        base.fill_(0x5A)
    return q


def _off(offsets):
    import torch
    return None if offsets is None else torch.from_numpy(offsets).to(DEV)


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])


def _zeros_behind(q):
    """The bytes from a row's end to the next multiple of 16."""
    import torch
    c = q.codes.view(torch.uint8)
    rows, cols = c.shape
    whole = -(-cols // 16) * 16
    wide = torch.as_strided(c, (rows, whole), (c.stride(0), 1), c.storage_offset())
    return wide[:, cols:].cpu().numpy()


# ---------------------------------------------------------------------------
# packing

PACK = [  # rows, cols, groups, format, pad, shift
    (1, 1, None, "e4m3", 0, 0), (1, 8, None, "e5m2", 0, 0), (3, 127, None, "e4m3", 1, 0), (128, 128, None, "e4m3", 0, 0),
    (129, 129, None, "e5m2", 0, 1), (5, 2880, None, "e4m3", 0, 0), (300, 200, None, "e4m3", 8, 8), (700, 72, 5, "e4m3", 0, 0),
    (333, 1000, 9, "e5m2", 3, 5), (64, 256, 40, "e4m3", 0, 0), (1000, 136, 130, "e4m3", 0, 0), (2, 16, 3, "e4m3", 0, 0),
]


@pytest.mark.parametrize("rows,cols,groups,fmt,pad,shift", PACK)
@pytest.mark.parametrize("which", ["both", "rows", "columns"])
def test_pack_bit_for_bit(rows, cols, groups, fmt, pad, shift, which):
    ve = _ve()
    print(f"[gpu] fp8 pack {rows}x{cols} groups {groups} {fmt} {which}", flush=True)
    rng = np.random.default_rng(rows * 1000 + cols)
    v = rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1))) * np.exp(2 * rng.standard_normal(cols))
    v.flat[0] = 0
    if rows > 4:
        v[1], v[2], v[3] = 0, v[2] * 1e-38, v[3] * 1e36   # zeros, next to both ends of the range
    bits = f64_to_bf16_bits(v)
    up = _up(bits)
    off = None if groups is None else group_offsets(rows, groups, rows + cols, first=min(1, rows - 1), spare=min(2, rows // 3))
    out, out_t = _filled(rows, cols, 1, fmt), _filled(cols, fp8.columns(rows, groups or 1), 1, fmt)
    ve.fp8_pack(_dev(bits, pad, shift), out if which != "columns" else None, out_t if which != "rows" else None,
                offsets=_off(off))
    if which != "columns":
        codes, e = fp8.pack(up, 1, fmt)
        got, ge = host(out)
        inside = np.zeros(rows, bool)
        for _, a, b in linear.parts(off, rows):
            inside[a:b] = True
        assert np.array_equal(got[inside], codes[inside]) and np.array_equal(ge[:, inside], e[:, inside])
        assert (got[~inside] == 0x5A).all() and (ge[:, ~inside] == 0x5A).all()
        assert not _zeros_behind(out)[inside].any()
    if which != "rows":
        t, used = fp8.transposed(up, off)
        codes, e = fp8.pack(t, 1, fmt)
        got, ge = host(out_t)
        assert np.array_equal(got[:, :used], codes[:, :used]) and np.array_equal(ge[:used // 128], e[:used // 128])
        assert (got[:, used:] == 0x5A).all() and (ge[used // 128:] == 0x5A).all()


@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_codes_of_every_bf16_value(fmt):
    """Every finite bf16 value as a block's largest, with values spread below it."""
    ve = _ve()
    amax = np.arange(0, 0x7F80, dtype=np.uint16)
    a = _up(amax)
    rng = np.random.default_rng(3)
    v = np.concatenate([a[:, None], -a[:, None], a[:, None] * rng.uniform(-1, 1, (len(a), 40)),
                        a[:, None] * np.exp(-rng.uniform(0, 14, (len(a), 40)))], 1)
    bits = f64_to_bf16_bits(v)
    bits[:, 0] = amax
    codes, e = fp8.pack(_up(bits), 1, fmt)
    out = _filled(*bits.shape, 1, fmt)
    ve.fp8_pack(_dev(bits), out)
    got, ge = host(out)
    assert np.array_equal(ge, e) and np.array_equal(got, codes)
    back = _dev(np.zeros_like(bits))
    ve.fp8_unpack(out, back)
    want = fp8.unpack(codes, e, 1, fmt)
    with np.errstate(over="ignore"):
        assert np.array_equal(_host(back), _up(f64_to_bf16_bits(want)))


@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_pack_of_non_finite_values(fmt):
    ve = _ve()
    v = np.random.default_rng(0).standard_normal((130, 140))
    v[0, 0], v[0, 1], v[1, 130], v[129, 5], v[7, 7] = np.inf, 3.0, -np.inf, np.nan, np.nan
    v[64, :128] = np.inf                                 # nothing finite in the block
    bits = f64_to_bf16_bits(np.where(np.isnan(v), 0, v))
    bits[np.isnan(v)] = 0x7FC0
    v = _up(bits)
    out, out_t = _filled(130, 140, 1, fmt), _filled(140, 256, 1, fmt)
    ve.fp8_pack(_dev(bits), out, out_t)
    codes, e = fp8.pack(v, 1, fmt)
    got, ge = host(out)
    same = (got == codes) | (np.isnan(v) & ((got & 127) == 127))
    assert same.all() and np.array_equal(ge, e)
    t, _ = fp8.transposed(v)
    codes, e = fp8.pack(t, 1, fmt)
    got, ge = host(out_t)
    assert ((got == codes) | (np.isnan(t) & ((got & 127) == 127))).all() and np.array_equal(ge, e)
    q, w = _filled(130, 140, 128, fmt), _dev(bits)
    ve.fp8_pack_weight(w, q)
    codes, e = fp8.pack(v, 128, fmt)
    got, ge = host(q)
    assert ((got == codes) | (np.isnan(v) & ((got & 127) == 127))).all() and np.array_equal(ge, e)


@pytest.mark.parametrize("name", linear.ACTS[1:])
@pytest.mark.parametrize("rows,cols,pad", [(200, 333, 0), (40, 256, 4), (131, 8, 1)])
def test_pack_of_a_gradient_through_an_activation(name, rows, cols, pad):
    """The value is within e32 = u |dz| + 2 A |dy| of dz (as the linear layer's
    dz), the block's exponent is the exact one's or, next to a border, its
    neighbour's, and a code is off by at most half a step: 2^-4 of the value or
    half the block's smallest step, 2^-10 2^e."""
    ve = _ve()
    dyb, zb = _bits((rows, cols), 1), f64_to_bf16_bits(2 * np.random.default_rng(2).standard_normal((rows, cols)))
    dy, z = _up(dyb), _up(zb)
    dz = dy * linear.slope(name, z)
    e32 = U * np.abs(dz) + (0 if name == "relu" else 2 * A) * np.abs(dy)
    out, out_t = _filled(rows, cols), _filled(cols, fp8.columns(rows))
    ve.fp8_pack(_dev(dyb, pad), out, out_t, z=_dev(zb, pad), activation=name)
    for q, ref, err in ((out, dz, e32), (out_t, fp8.transposed(dz)[0], fp8.transposed(e32)[0])):
        c, e = host(q)
        _, ee = fp8.pack(ref, 1)
        assert (np.abs(e.astype(int) - ee.astype(int)) <= 1).all()
        step = np.repeat(2.0 ** (np.maximum(e, ee).astype(float) - 127).T, 128, 1)[:, :ref.shape[1]]
        _within(fp8.unpack(c, e), ref, err + np.maximum(2.0 ** -4 * (np.abs(ref) + err), 2.0 ** -10 * step) + TINY, name)


@pytest.mark.parametrize("groups,rows,cols,fmt,pad,shift", [
    (None, 1, 1, "e4m3", 0, 0), (None, 128, 128, "e4m3", 0, 0), (None, 300, 200, "e5m2", 3, 1), (3, 136, 264, "e4m3", 0, 0),
    (2, 65, 1000, "e4m3", 8, 8), (5, 257, 17, "e4m3", 0, 0), (None, 2880, 72, "e4m3", 0, 0),
])
def test_pack_weight_bit_for_bit(groups, rows, cols, fmt, pad, shift):
    ve = _ve()
    print(f"[gpu] fp8 weights {groups}x{rows}x{cols} {fmt}", flush=True)
    shape = (rows, cols) if groups is None else (groups, rows, cols)
    bits = _bits(shape, rows + cols, 1.0)
    codes, e, _ = packed_values(_up(bits), 128, fmt)
    for which in ("both", "rows", "columns"):
        out, out_t = _filled(rows, cols, 128, fmt, groups), _filled(cols, rows, 128, fmt, groups)
        ve.fp8_pack_weight(_dev(bits, pad, shift), out if which != "columns" else None, out_t if which != "rows" else None)
        if which != "columns":
            got, ge = host(out)
            assert np.array_equal(got, codes) and np.array_equal(ge, e)
            if groups is None:
                assert not _zeros_behind(out).any()
        if which != "rows":
            got, ge = host(out_t)
            assert np.array_equal(got, np.swapaxes(codes, -1, -2)) and np.array_equal(ge, np.swapaxes(e, -1, -2))
            if groups is None:
                assert not _zeros_behind(out_t).any()


@pytest.mark.parametrize("rows,cols,block,fmt,pad,shift", [
    (1, 1, 1, "e4m3", 0, 0), (130, 257, 1, "e5m2", 0, 1), (130, 257, 128, "e4m3", 1, 0), (33, 1024, 1, "e4m3", 8, 8)])
def test_unpack(rows, cols, block, fmt, pad, shift):
    """Every code under exponents over the whole range (255: NaN)."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(rows + cols)
    codes = rng.integers(0, 256, (rows, cols)).astype(np.uint8)
    e = rng.integers(0, 256, (-(-cols // 128), -(-rows // block))).astype(np.uint8)
    e.flat[0] = 255
    out = _dev(np.zeros((rows, cols), np.uint16), pad, shift)
    ve.fp8_unpack(device(codes, e, block, fmt, pad), out)
    torch.cuda.synchronize()
    got = out.float().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        want = fp8.unpack(codes, e, block, fmt).astype(np.float32)
        # one rounding to bf16, by torch on the host
        ref = torch.from_numpy(want).to(torch.bfloat16).float().numpy()
    assert np.array_equal(got, ref, equal_nan=True)


def test_unpack_of_groups():
    import torch
    ve = _ve()
    rng = np.random.default_rng(5)
    codes, e = rng.integers(0, 126, (3, 200, 130)).astype(np.uint8), rng.integers(100, 150, (3, 2, 2)).astype(np.uint8)
    out = torch.full((3, 200, 136), 7.0, dtype=torch.bfloat16, device=DEV)
    ve.fp8_unpack(device(codes, e, 128, pad=1), out[..., :130])
    got = _host(out)
    assert np.array_equal(got[..., :130], np.stack([fp8.unpack(c, x, 128) for c, x in zip(codes, e)]))
    assert (got[..., 130:] == 7).all()


# ---------------------------------------------------------------------------
# products

def _forward(case, seed=0, **kw):
    import torch
    ve = _ve()
    T, K, N, E, name, bias, res, zout, fmt, pad = case
    print(f"[gpu] fp8 forward {case}", flush=True)
    rng = np.random.default_rng(seed + T + K + N)
    off = None if E is None else group_offsets(T, E, seed + T, first=min(1, T - 1), spare=min(2, T // 3))
    xc, xe, x = packed_values(rng.standard_normal((T, K)) * np.exp(2 * rng.standard_normal((T, 1))), 1, fmt)
    w = rng.standard_normal((N, K) if E is None else (E, N, K)) * K ** -0.5 * np.exp(rng.standard_normal((N, 1)))
    wc, we, w = packed_values(w, 128, "e4m3")
    bb = _bits((N,) if E is None else (E, N), 5) if bias else None
    rb = _bits((T, N), 6) if res else None
    ref_y, ref_z, mag = linear.forward(x, w, None if bb is None else _up(bb), name, None if rb is None else _up(rb), off)
    y = torch.full((T, N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    z = torch.full((T, N + pad), 7.0, dtype=torch.bfloat16, device=DEV) if zout else None
    r = None if rb is None else _dev(rb)
    if res == "in place":
        y[:, :N].copy_(r)
        r = y[:, :N]
    ve.fp8_linear_forward(device(xc, xe, 1, fmt, pad % 3), device(wc, we, 128, pad=pad % 2), y[:, :N],
                          bias=None if bb is None else torch.from_numpy(bb.view(np.int16)).to(DEV),
                          activation=name, residual=r, z=None if z is None else z[:, :N], offsets=_off(off), **kw)
    bz, by = forward_bounds(ref_y, ref_z, mag, cut_rows(x, w, off), K, name, rb)
    inside = np.zeros(T, bool)
    for _, a, b in linear.parts(off, T):
        inside[a:b] = True
    got = _host(y)
    _within(got[inside, :N], ref_y[inside], by[inside], "y")
    assert (got[:, N:] == 7).all()
    if res != "in place":
        assert (got[~inside, :N] == 7).all()
    if z is not None:
        gz = _host(z)
        _within(gz[inside, :N], ref_z[inside], bz[inside], "z")
        assert (gz[:, N:] == 7).all() and (gz[~inside, :N] == 7).all()
    return y


FORWARD = [  # tokens, in, out, groups, activation, bias, residual, z, format of x, pad
    (1, 1, 1, None, "none", False, None, False, "e4m3", 0),
    (1, 8192, 40, None, "none", True, None, False, "e4m3", 0),
    (2, 130, 264, None, "silu", True, "apart", True, "e5m2", 0),
    (5, 1000, 257, None, "gelu", False, "in place", False, "e4m3", 3),
    (16, 256, 128, None, "none", False, None, False, "e4m3", 8),
    (17, 384, 72, None, "gelu_tanh", True, None, True, "e4m3", 0),
    (33, 2880, 128, None, "none", True, "apart", False, "e4m3", 0),
    (129, 128, 129, None, "relu", True, None, True, "e5m2", 1),
    (200, 127, 300, None, "none", False, "in place", False, "e4m3", 0),
    (257, 640, 513, None, "silu", False, None, True, "e4m3", 8),
    (300, 72, 264, 4, "none", True, None, False, "e4m3", 0),
    (64, 300, 200, 40, "silu", True, "apart", True, "e5m2", 0),
    (700, 256, 136, 9, "none", False, None, False, "e4m3", 8),
    (5, 512, 64, 200, "none", True, None, False, "e4m3", 0),
    (600, 1024, 520, 3, "gelu", False, "apart", False, "e4m3", 0),
]


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    _forward(case)


@pytest.mark.parametrize("path,split", [(2, 0), (2, 1), (3, 0), (3, 1), (4, 1)])
@pytest.mark.parametrize("case", [
    (70, 4096, 264, None, "silu", True, None, True, "e4m3", 0),
    (300, 2056, 520, None, "none", True, "in place", False, "e5m2", 8),
    (129, 1000, 257, None, "gelu", False, "apart", False, "e4m3", 1),
    (700, 384, 136, 9, "relu", True, None, True, "e4m3", 0),
    (900, 640, 264, 70, "none", True, "apart", False, "e4m3", 0),
], ids=lambda c: "-".join(map(str, c)))
def test_forward_forms(case, path, split):
    with _ve().options(linear_path=path, linear_split=split):
        _forward(case, seed=1)


def _backward(case, seed=0, accumulate=False, dx=True, dw=True):
    import torch
    ve = _ve()
    T, K, N, E, add, wide, fmt, pad = case
    print(f"[gpu] fp8 backward {case}", flush=True)
    rng = np.random.default_rng(seed + T + K + N)
    off = None if E is None else group_offsets(T, E, seed + T, first=min(1, T - 1), spare=min(2, T // 3))
    dy0 = 1e-3 * rng.standard_normal((T, N)) * np.exp(rng.standard_normal((T, 1)))
    x0 = rng.standard_normal((T, K)) * np.exp(rng.standard_normal(K))
    w0 = rng.standard_normal((N, K) if E is None else (E, N, K)) * K ** -0.5
    dyc, dye, dy = packed_values(dy0, 1, fmt)
    wc, we, wt = packed_values(np.ascontiguousarray(np.swapaxes(w0, -1, -2)), 128, "e4m3")
    dytc, dyte, dyt = packed_values(fp8.transposed(dy0, off)[0], 1, fmt)
    xtc, xte, xt = packed_values(fp8.transposed(x0, off)[0], 1, "e4m3")
    addb = _bits((T, K), 3) if add else None
    ref = linear.backward(dy, np.swapaxes(wt, -1, -2), None, None, "none", None if addb is None else _up(addb), off)["dx"]
    mag = linear.backward(np.abs(dy), np.abs(np.swapaxes(wt, -1, -2)), offsets=off)["dx"]
    ref_w, mag_w = fp8.weight_gradient(dyt, xt, off, T)
    gdx = torch.full((T, K + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    shape = (*(() if E is None else (E,)), N, K + pad)
    gdw = torch.full(shape, 7.0, dtype=torch.float32 if wide else torch.bfloat16, device=DEV)
    held = None
    if accumulate:
        held = rng.standard_normal((*shape[:-1], K))
        gdw[..., :K] = torch.from_numpy(held).to(gdw.dtype).to(DEV)
        held = _host(gdw)[..., :K]
    r = None if addb is None else _dev(addb)
    if add == "in place":
        gdx[:, :K].copy_(r)
        r = gdx[:, :K]
    ve.fp8_linear_backward(dy=device(dyc, dye, 1, fmt) if dx else None, w_t=device(wc, we, 128, pad=1) if dx else None,
                           dx=gdx[:, :K] if dx else None, dx_add=r if dx else None,
                           dy_t=device(dytc, dyte, 1, fmt, pad % 2) if dw else None, x_t=device(xtc, xte) if dw else None,
                           dw=gdw[..., :K] if dw else None, accumulate=accumulate, offsets=_off(off), tokens=T)
    inside = np.zeros(T, bool)
    for _, a, b in linear.parts(off, T):
        inside[a:b] = True
    got = _host(gdx)
    if dx:
        bound = gamma(N + 2) * mag + cut_rows(dy, wt, off) + TINY
        if add:
            bound = bound + U * (np.abs(ref) + bound)
        _within(got[inside, :K], ref[inside], rounded(bound, ref)[inside], "dx")
        assert (got[:, K:] == 7).all() and (add == "in place" or (got[~inside, :K] == 7).all())
    else:
        assert (got == 7).all()
    got = _host(gdw)
    if dw:
        bound = gamma(T + 130) * mag_w + TINY
        if not wide:
            at = 0
            for e, a, b in linear.parts(off, T):
                n = at + -(-(b - a) // 128) * 128
                bound[... if off is None else e] += cut(dyt[:, at:n], xt[:, at:n])
                at = n
        if held is not None:
            ref_w = ref_w + held
            bound = bound + U * (np.abs(ref_w) + bound)
        _within(got[..., :K], ref_w, bound if wide else rounded(bound, ref_w), "dw")
        assert (got[..., K:] == 7).all()
    else:
        assert (got == 7).all()


BACKWARD = [  # tokens, in, out, groups, dx_add, fp32 dw, format of dy, pad
    (1, 1, 1, None, None, False, "e4m3", 0),
    (1, 300, 77, None, None, True, "e5m2", 0),
    (20, 128, 2880, None, "apart", False, "e4m3", 0),
    (130, 257, 129, None, "in place", True, "e4m3", 1),
    (500, 264, 520, None, None, False, "e5m2", 8),
    (300, 72, 264, 4, "apart", True, "e4m3", 0),
    (64, 300, 200, 40, None, False, "e5m2", 3),
    (900, 512, 136, 5, None, True, "e4m3", 8),
    (5, 256, 64, 100, None, True, "e4m3", 0),
    (2000, 136, 128, None, None, True, "e4m3", 0),
]


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward(case, accumulate):
    _backward(case, accumulate=accumulate)


@pytest.mark.parametrize("path,split", [(2, 0), (2, 1), (3, 0), (3, 1)])
@pytest.mark.parametrize("case", [
    (4000, 136, 264, None, "apart", False, "e4m3", 0),
    (3000, 72, 136, None, None, True, "e5m2", 8),
    (2500, 129, 65, None, "in place", False, "e4m3", 1),
    (700, 264, 392, 9, None, False, "e5m2", 0),
    (900, 136, 264, 70, "apart", False, "e4m3", 0),
    (800, 136, 264, 70, None, True, "e4m3", 0),
], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_forms(case, path, split, accumulate):
    with _ve().options(linear_path=path, linear_split=split):
        _backward(case, seed=1, accumulate=accumulate)


def test_backward_outputs_are_optional():
    _backward((300, 72, 264, 4, None, True, "e4m3", 0), dx=False)
    _backward((300, 72, 264, 4, None, True, "e4m3", 0), dw=False)
    _backward((100, 72, 64, None, None, False, "e5m2", 0), dx=False)
    _ve().fp8_linear_backward()


def test_no_tokens_and_empty_groups():
    import torch
    ve = _ve()
    w = ve.new_fp8(24, 40, 128, groups=3, device=DEV)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    y = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    ve.fp8_linear_forward(ve.new_fp8(0, 40, device=DEV), w, y, offsets=off)
    dw = torch.full((3, 24, 40), 3.0, device=DEV)
    none = dict(dy_t=ve.new_fp8(24, 0, device=DEV), x_t=ve.new_fp8(40, 0, device=DEV), dw=dw, offsets=off, tokens=0)
    ve.fp8_linear_backward(**none, accumulate=True)
    assert bool((dw == 3).all())
    ve.fp8_linear_backward(**none)
    assert bool((dw == 0).all())
    ve.fp8_pack(torch.empty(0, 40, dtype=torch.bfloat16, device=DEV), ve.new_fp8(0, 40, device=DEV))


def test_zeros_times_a_large_scale_and_nan_rows():
    """A block of NaN codes makes its row of y NaN and no other; a block of
    zeros adds nothing whatever its exponent."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(0)
    xc, xe, x = packed_values(rng.standard_normal((40, 300)), 1, "e4m3")
    wc, we, w = packed_values(rng.standard_normal((70, 300)), 128, "e4m3")
    xc[3, 5] = 0x7F
    xc[7, 128:256], xe[1, 7] = 0, 240
    xe[2, 9] = 255
    y = torch.empty(40, 70, dtype=torch.bfloat16, device=DEV)
    ve.fp8_linear_forward(device(xc, xe), device(wc, we, 128), y)
    x = fp8.unpack(xc, xe)
    got = _host(y)
    bad = np.zeros(40, bool)
    bad[[3, 9]] = True
    assert np.isnan(got[bad]).all()
    ref, z, mag = linear.forward(x[~bad], w)
    _within(got[~bad], ref, forward_bounds(ref, z, mag, cut(x[~bad], w), 300, "none")[1], "y")


def test_powers_at_the_ends_of_the_range():
    """Exponents of both operands far from 0 that cancel in the product."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(1)
    xc, xe, x = packed_values(rng.standard_normal((20, 256)), 1, "e4m3")
    wc, we, w = packed_values(rng.standard_normal((30, 256)), 128, "e4m3")
    ref, z, mag = linear.forward(x, w)
    for shift in (-100, -40, 40, 100):
        y = torch.empty(20, 30, dtype=torch.bfloat16, device=DEV)
        ve.fp8_linear_forward(device(xc, (xe.astype(int) + shift)), device(wc, (we.astype(int) - shift), 128), y)
        _within(_host(y), ref, forward_bounds(ref, z, mag, cut(x, w), 256, "none")[1], shift)


def test_gradients_are_difference_quotients():
    """On whole numbers of few bits every value here is exact (products and
    their sums below 2^8 in bf16 outputs), and so are the differences."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(4)
    T, K, N = 6, 20, 12
    x, w = rng.integers(-2, 3, (T, K)).astype(float), rng.integers(-1, 2, (N, K)).astype(float)
    dy = rng.integers(-2, 3, (T, N)).astype(float)

    def q(v, block=1):
        out = ve.new_fp8(*v.shape, block, device=DEV)
        t = torch.from_numpy(v).to(torch.bfloat16).to(DEV)
        if block == 1:
            ve.fp8_pack(t, out)
        else:
            ve.fp8_pack_weight(t, out)
        return out

    def loss(x, w):
        y = torch.empty(len(x), N, dtype=torch.bfloat16, device=DEV)
        ve.fp8_linear_forward(q(x), q(w, 128), y)
        return (y.double().cpu().numpy() * dy).sum()

    w_t, dyt, xt = (ve.new_fp8(K, N, 128, device=DEV), ve.new_fp8(N, 128, device=DEV), ve.new_fp8(K, 128, device=DEV))
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).to(DEV)  # noqa: E731
    ve.fp8_pack_weight(dev(w), None, w_t)
    ve.fp8_pack(dev(x), None, xt)
    dyq = ve.new_fp8(T, N, device=DEV)
    ve.fp8_pack(dev(dy), dyq, dyt)
    dx, dw = torch.empty(T, K, dtype=torch.bfloat16, device=DEV), torch.empty(N, K, device=DEV)
    ve.fp8_linear_backward(dy=dyq, w_t=w_t, dx=dx, dy_t=dyt, x_t=xt, dw=dw)
    for v, g, other in ((x, _host(dx), False), (w, _host(dw), True)):
        for i in list(np.ndindex(v.shape))[::7]:
            d = np.zeros_like(v)
            d[i] = 1
            diff = (loss(x, w + d) - loss(x, w - d)) / 2 if other else (loss(x + d, w) - loss(x - d, w)) / 2
            assert diff == g[i], (i, diff, g[i])


def test_bad_offsets_stay_inside_the_buffers():
    """Offsets outside the rules: any values, but no access outside (the
    buffers' surroundings are kept)."""
    import torch
    ve = _ve()
    T, K, N = 300, 200, 136
    rng = np.random.default_rng(0)
    x, dy = _dev(_bits((T, K), 0)), _dev(_bits((T, N), 1))
    wc, we, _ = packed_values(rng.standard_normal((4, N, K)), 128, "e4m3")
    wtc, wte, _ = packed_values(rng.standard_normal((4, K, N)), 128, "e4m3")
    for bad in ([-5, 900, 20, -1, 10 ** 12], [300, 0, 300, 0, 300], [0, 300, 300, 299, 305], [-(10 ** 18)] * 5):
        off = torch.tensor(bad, dtype=torch.int64, device=DEV)
        xq, xt = ve.new_fp8(T, K, device=DEV), ve.new_fp8(K, fp8.columns(T, 4), device=DEV)
        dq, dt = ve.new_fp8(T, N, device=DEV), ve.new_fp8(N, fp8.columns(T, 4), device=DEV)
        ve.fp8_pack(x, xq, xt, offsets=off)
        ve.fp8_pack(dy, dq, dt, offsets=off)
        y = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
        dx = torch.full((T + 2, K), 7.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((6, N, K), 7.0, device=DEV)
        ve.fp8_linear_forward(xq, device(wc, we, 128), y[1:-1], offsets=off)
        ve.fp8_linear_backward(dy=dq, w_t=device(wtc, wte, 128), dx=dx[1:-1], dy_t=dt, x_t=xt, dw=dw[1:-1], offsets=off)
        torch.cuda.synchronize()
        assert all(bool((t[0] == 7).all()) and bool((t[-1] == 7).all()) for t in (y, dx, dw))


# ---------------------------------------------------------------------------
# how calls may be made

def _layer(T=700, K=264, N=392, E=5, seed=0):
    """A grouped layer's calls from bf16 on, and their outputs."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(seed)
    off = _off(group_offsets(T, E, seed, first=1, spare=2))
    x, dy, z = (_dev(_bits((T, n), seed + i)) for i, n in enumerate((K, N, N)))
    w = _dev(_bits((E, N, K), seed + 9))
    q = dict(x8=ve.new_fp8(T, K, device=DEV), dy8=ve.new_fp8(T, N, device=DEV), w8=ve.new_fp8(N, K, 128, groups=E, device=DEV),
             w8t=ve.new_fp8(K, N, 128, groups=E, device=DEV), xt=ve.new_fp8(K, fp8.columns(T, E), device=DEV),
             dyt=ve.new_fp8(N, fp8.columns(T, E), device=DEV))
    y, dx = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV), torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    dw, dw32 = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV), torch.zeros(E, N, K, device=DEV)
    back = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)

    def call(**kw):
        ve.fp8_pack(x, q["x8"], q["xt"], offsets=off, **kw)
        ve.fp8_pack(dy, q["dy8"], q["dyt"], z=z, activation="silu", offsets=off, **kw)
        ve.fp8_pack_weight(w, q["w8"], q["w8t"], **kw)
        ve.fp8_unpack(q["x8"], back, **kw)
        ve.fp8_linear_forward(q["x8"], q["w8"], y, activation="gelu", offsets=off, **kw)
        for d in (dw, dw32):
            ve.fp8_linear_backward(dy=q["dy8"], w_t=q["w8t"], dx=dx, dy_t=q["dyt"], x_t=q["xt"], dw=d, offsets=off, **kw)

    outs = [y, dx, dw, dw32, back] + [t for v in q.values() for t in (v.codes.view(torch.uint8), v.scales)]
    return call, outs


def test_same_bits_every_call_and_on_other_streams():
    import torch
    call, outs = _layer()
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream(DEV)
    for stream in (None, s, s.cuda_stream):
        for t in outs:
            t.fill_(0)
        s.wait_stream(torch.cuda.current_stream())
        call(stream=stream)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    import torch
    pairs = [_layer(seed=3) for _ in range(2)]
    pairs[0][0]()
    torch.cuda.synchronize()
    want = [t.clone() for t in pairs[0][1]]
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for t in pairs[0][1]:
        t.fill_(0)
    torch.cuda.synchronize()
    for _ in range(5):
        for (call, _), s in zip(pairs, streams):
            call(stream=s)
    torch.cuda.synchronize()
    for _, outs in pairs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_captured_graph_replays():
    import torch
    call, outs = _layer(seed=5)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in outs:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        call()                                             # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_split_products_need_and_take_their_workspace():
    import torch
    ve = _ve()
    rng = np.random.default_rng(0)
    T, K, N = 200, 8192, 264
    xc, xe, x = packed_values(rng.standard_normal((T, K)), 1, "e4m3")
    wc, we, w = packed_values(rng.standard_normal((N, K)), 128, "e4m3")
    xq, wq = device(xc, xe), device(wc, we, 128)
    y = torch.full((T, N), 5.0, dtype=torch.bfloat16, device=DEV)
    need = ve.fp8_linear_forward_workspace(xq, wq, y)
    assert need > 0
    for ws in (torch.empty(need - 256, dtype=torch.uint8, device=DEV), torch.empty(need + 256, dtype=torch.uint8, device=DEV)[16:]):
        with pytest.raises(ve.VeError, match="workspace"):
            ve.fp8_linear_forward(xq, wq, y, workspace=ws)
    torch.cuda.synchronize()
    assert bool((y == 5).all())
    ve.fp8_linear_forward(xq, wq, y, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    ref, z, mag = linear.forward(x, w)
    _within(_host(y), ref, forward_bounds(ref, z, mag, cut(x, w), K, "none")[1], "y")
    dw = torch.empty(40, 72, device=DEV)
    assert ve.fp8_linear_backward_workspace(dy_t=ve.new_fp8(40, 8192, device=DEV), x_t=ve.new_fp8(72, 8192, device=DEV), dw=dw,
                                            tokens=8192) > 0


def test_offsets_beyond_32_bits():
    """Codes, outputs and weights past 4 GiB: the last group's rows."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(0)
    K, N, E = 8192, 8192, 66                               # 4.4 GB of weights
    w8 = ve.new_fp8(N, K, 128, groups=E, device=DEV)
    wc, we, w = packed_values(rng.standard_normal((N, 128)), 128, "e4m3")
    w8.codes[E - 1].view(torch.uint8)[:, -128:] = torch.from_numpy(wc).to(DEV)
    w8.scales[E - 1][-1, :] = torch.from_numpy(we[0]).to(DEV)
    for T in (20, 700):                                    # few rows, and tiles
        off = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
        off[E] = T
        xc, xe, x = packed_values(rng.standard_normal((T, K)), 1, "e4m3")
        y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
        ve.fp8_linear_forward(device(xc, xe), w8, y, offsets=off)
        ref, z, mag = linear.forward(x[:, -128:], w)
        _within(_host(y), ref, forward_bounds(ref, z, mag, cut(x[:, -128:], w), 128, "none")[1], T)
    back = torch.empty(E, 512, K, dtype=torch.bfloat16, device=DEV)
    ve.fp8_unpack(ve.Fp8(w8.codes[:, -512:], w8.scales[..., -4:], 128), back)
    assert np.array_equal(_host(back[-1, :, -128:]), w[-512:])
    del back
    # dw of the last group, 4.4 G elements of 2 bytes from the first one's
    dw = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    off[E] = 40
    dy, xx = rng.standard_normal((40, N)), rng.standard_normal((40, K))
    dyc, dye, dyv = packed_values(fp8.transposed(dy, off.cpu().numpy())[0], 1, "e4m3")
    xtc, xte, xv = packed_values(fp8.transposed(xx, off.cpu().numpy())[0], 1, "e4m3")
    ve.fp8_linear_backward(dy_t=device(dyc, dye), x_t=device(xtc, xte), dw=dw, offsets=off, tokens=40)
    ref, mag = dyv[:64, :128] @ xv[:, :128].T, np.abs(dyv[:64, :128]) @ np.abs(xv[:, :128]).T
    _within(_host(dw[-1, :64]), ref, rounded(gamma(170) * mag + cut(dyv[:64], xv) + TINY, ref), "dw")
    assert bool((dw[:-1:13] == 0).all())
    del dw, w8
    # rows of 4.8 GB
    T, K, N = 600000, 8192, 72
    x8, y = ve.new_fp8(T, K, device=DEV), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    xb, wb = _bits((300, K), 1), _bits((N, K), 2)
    big = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    big[-300:] = _dev(xb)
    ve.fp8_pack(big, x8)
    del big
    w8 = ve.new_fp8(N, K, 128, device=DEV)
    ve.fp8_pack_weight(_dev(wb), w8)
    ve.fp8_linear_forward(x8, w8, y)
    xv, wv = packed_values(_up(xb), 1, "e4m3")[2], packed_values(_up(wb), 128, "e4m3")[2]
    ref, z, mag = linear.forward(xv, wv)
    _within(_host(y[-300:]), ref, forward_bounds(ref, z, mag, cut(xv, wv), K, "none")[1], "rows")
    assert bool((y[:-300:997] == 0).all())


def test_binding_refuses_rows_without_room():
    """The last row's memory has to go on to whole 16 bytes (scales: 4)."""
    import torch
    ve = _ve()
    c = torch.zeros(4 * 112, dtype=torch.uint8, device=DEV)[:3 * 112 + 100].view(torch.float8_e4m3fn)
    short = torch.empty(3 * 112 + 100, dtype=torch.uint8, device=DEV)
    good = ve.new_fp8(4, 100, device=DEV)
    out = torch.empty(4, 100, dtype=torch.bfloat16, device=DEV)
    ve.fp8_unpack(good, out)
    short = torch.as_strided(short.view(torch.float8_e4m3fn), (4, 100), (112, 1))
    with pytest.raises(ValueError, match="memory"):
        ve.fp8_unpack(ve.Fp8(short, good.scales), out)
    with pytest.raises(ve.VeError, match="16 bytes"):
        ve.fp8_unpack(ve.Fp8(torch.zeros(4, 100, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, :96],
                             ve.new_fp8(4, 96, device=DEV).scales), out[:, :96])
    del c


def test_more_workgroups_than_the_few_row_form_may_have():
    """40,000 groups of one row each and 4,096 columns: 10 million workgroups of
    512 threads would pass a grid's 2^32 threads, so the tiles take it."""
    import torch
    ve = _ve()
    E, N, K = 40000, 4096, 16
    w8 = ve.new_fp8(N, K, 128, groups=E, device=DEV)
    w8.codes.view(torch.uint8).fill_(0x38)                 # 1.0
    w8.scales.fill_(127)
    x = torch.arange(E, device=DEV).remainder(16).to(torch.bfloat16)[:, None].expand(E, K).contiguous()
    x8, y = ve.new_fp8(E, K, device=DEV), torch.zeros(E, N, dtype=torch.bfloat16, device=DEV)
    ve.fp8_pack(x, x8)
    ve.fp8_linear_forward(x8, w8, y, offsets=torch.arange(E + 1, device=DEV))
    assert torch.equal(y, (x[:, :1] * K).expand(E, N))
