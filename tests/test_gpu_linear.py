"""GPU results of the linear layer's operators and of 8-bit saved activations
against the fp64 oracle (oracle/linear.py), within the elementwise bounds of
tests/linear_common.py; the 8-bit code bit for bit."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import linear
from oracle.muon import bf16_bits_to_f64, f64_to_bf16_bits
from linear_common import backward_bounds, forward_bounds, group_offsets

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _bits(shape, seed, scale=1.0):
    return f64_to_bf16_bits(np.random.default_rng(seed).standard_normal(shape) * scale)


def _up(bits):
    return bf16_bits_to_f64(bits).reshape(bits.shape)


def _dev(bits, pad=0, shift=0):
    """A device copy whose rows are `pad` elements longer than needed and
    start `shift` elements into an allocation (NaN around them)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    rows, cols = t.numel() // t.shape[-1], t.shape[-1]
    if not pad and not shift:
        return t.to(DEV).view(torch.bfloat16)
    flat = torch.full((shift + rows * (cols + pad) + 64,), 0x7FC0, dtype=torch.int16)
    flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = t.reshape(rows, cols)
    strides = [cols + pad, 1] if t.dim() == 2 else [t.shape[1] * (cols + pad), cols + pad, 1]
    return torch.as_strided(flat.to(DEV), t.shape, strides if t.dim() > 1 else [1], shift).view(torch.bfloat16)


def _out(shape, dtype="bfloat16", pad=0, shift=0):
    """An output buffer (filled with a marker) with padded, shifted rows."""
    import torch
    dt = getattr(torch, dtype)
    rows, cols = int(np.prod(shape[:-1])), shape[-1]
    flat = torch.full((shift + rows * (cols + pad) + 64,), 7.0, dtype=dt, device=DEV)
    strides = [cols + pad, 1] if len(shape) < 3 else [shape[-2] * (cols + pad), cols + pad, 1]
    v = torch.as_strided(flat, shape, strides[-len(shape):], shift)
    return v, flat


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _untouched(flat, view):
    """Everything around the view still holds the marker."""
    import torch
    mark = torch.full_like(flat, 7.0)
    torch.as_strided(mark, view.shape, view.stride(), view.storage_offset()).copy_(view)
    return torch.equal(mark.view(torch.int16 if flat.element_size() == 2 else torch.int32),
                       flat.view(torch.int16 if flat.element_size() == 2 else torch.int32))


def _within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])


# ---------------------------------------------------------------------------
# 8-bit saved activations

@pytest.mark.parametrize("rows,cols,block,pad,shift", [
    (1, 1, 32, 0, 0), (1, 31, 32, 0, 0), (3, 33, 32, 0, 0), (5, 128, 128, 0, 0), (7, 129, 128, 0, 0),
    (64, 2880, 64, 0, 0), (33, 1000, 128, 8, 8), (17, 257, 64, 3, 1), (1000, 72, 32, 0, 0), (2, 20000, 128, 0, 5),
])
def test_pack_and_unpack_bit_for_bit(rows, cols, block, pad, shift):
    import torch
    ve = _ve()
    print(f"[gpu] act8 {rows}x{cols} block {block} pad {pad} shift {shift}", flush=True)
    rng = np.random.default_rng(rows * 1000 + cols)
    v = rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1)))
    v.flat[0] = 0
    if rows > 2:
        v[1] = 0                                     # a row of zeros
        v[2, : min(cols, block)] *= 1e-38            # a run below 2^-100
    bits = f64_to_bf16_bits(v)
    codes, scales = linear.pack(_up(bits).astype(np.float32), block)
    x = _dev(bits, pad, shift)
    c = torch.full((rows, cols + pad), 99, dtype=torch.int8, device=DEV)
    s = torch.full((rows, -(-cols // block) + 1), 7.0, device=DEV)
    q = ve.Act8(c[:, :cols], s[:, :-1], block)
    ve.act8_pack(x, q)
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert bool((c[:, cols:] == 99).all()) and bool((s[:, -1] == 7).all())
    out, flat = _out((rows, cols), pad=pad, shift=shift)
    ve.act8_unpack(q, out)
    want = f64_to_bf16_bits(linear.unpack(codes, scales, block).astype(np.float64))
    got = out.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.array_equal(got, want.reshape(got.shape))
    assert _untouched(flat, out)


def test_scales_of_every_bf16_magnitude():
    """One run for each positive finite bf16 value as its largest magnitude
    (normal and subnormal), with values spread below it: scales and codes bit
    for bit, in waves of one kind and in mixed ones."""
    import torch
    ve = _ve()
    amax = np.arange(1, 0x7F80, dtype=np.uint16)
    for order in (np.arange(len(amax)), np.random.default_rng(0).permutation(len(amax))):
        a = bf16_bits_to_f64(amax[order])
        v = a[:, None] * np.random.default_rng(1).uniform(-1, 1, (len(a), 32))
        v[:, 7] = a
        v[:, 8] = -a / 2
        bits = f64_to_bf16_bits(v)
        codes, scales = linear.pack(_up(bits).astype(np.float32), 32)
        q = ve.new_act8(len(a), 32, 32, DEV)
        ve.act8_pack(_dev(bits), q)
        torch.cuda.synchronize()
        assert np.array_equal(q.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
        assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_pack_of_non_finite_runs():
    import torch
    ve = _ve()
    v = np.random.default_rng(1).standard_normal((6, 96))
    bits = f64_to_bf16_bits(v)
    bits[0, 3], bits[1, 40], bits[2, 95], bits[3, 0] = 0x7F80, 0xFF80, 0x7FC0, 0xFFFF
    bits[4, 10:12] = 0x7F7F                                  # the largest finite value
    codes, scales = linear.pack(_up(bits).astype(np.float32), 32)
    q = ve.new_act8(6, 96, 32, DEV)
    ve.act8_pack(_dev(bits), q)
    out = torch.empty(6, 96, dtype=torch.bfloat16, device=DEV)
    ve.act8_unpack(q, out)
    torch.cuda.synchronize()
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales, equal_nan=True)
    nan = torch.isnan(out).cpu().numpy()
    for r, run in ((0, 0), (1, 1), (2, 2), (3, 0)):
        assert nan[r, 32 * run:32 * run + 32].all()
    assert nan.sum() == 4 * 32


# ---------------------------------------------------------------------------
# forward

FORWARD = [
    # T, K, N, groups, act, bias, residual, z, block, pad, shift
    (1, 1, 1, None, "none", False, False, False, 0, 0, 0),
    (1, 8192, 1024, None, "none", True, False, False, 0, 0, 0),
    (1, 64, 8, None, "silu", True, True, True, 0, 0, 0),
    (3, 7, 5, None, "gelu", True, True, True, 32, 0, 0),
    (16, 128, 96, None, "relu", False, True, False, 0, 0, 0),
    (17, 2880, 200, None, "gelu_tanh", True, False, True, 0, 0, 0),
    (33, 72, 1000, None, "none", True, True, False, 0, 8, 8),
    (64, 520, 264, None, "silu", True, False, False, 0, 0, 0),
    (65, 520, 264, None, "silu", True, False, False, 64, 0, 0),
    (127, 200, 129, None, "gelu", True, True, True, 128, 1, 3),
    (130, 1000, 1160, None, "relu", False, False, False, 128, 0, 0),
    (256, 64, 256, None, "none", False, False, False, 0, 0, 0),
    (300, 136, 520, None, "gelu_tanh", True, True, True, 32, 8, 0),
    (40, 136, 264, 1, "silu", True, False, True, 64, 0, 0),
    (40, 136, 264, 5, "none", True, True, False, 0, 0, 0),
    (333, 264, 392, 7, "gelu", True, True, True, 128, 0, 0),
    (333, 99, 75, 7, "silu", True, True, True, 32, 3, 1),
    (700, 64, 136, 70, "relu", True, False, False, 0, 0, 0),
    (200, 80, 72, 130, "none", False, False, False, 0, 8, 0),
]


def _forward_case(T, K, N, E, name, has_bias, has_res, has_z, block, pad, shift, seed=0):
    import torch
    ve = _ve()
    off = None if E is None else group_offsets(T, E, seed + E, first=2 if T > 20 else 0, spare=3 if T > 20 else 0)
    xb = _bits((T, K), seed + 1)
    wb = _bits((N, K) if E is None else (E, N, K), seed + 2, K ** -0.5)
    bb = _bits((N,) if E is None else (E, N), seed + 3) if has_bias else None
    rb = _bits((T, N), seed + 4) if has_res else None
    up = lambda v: None if v is None else _up(v)  # noqa: E731
    y, z, mag = linear.forward(up(xb), up(wb), up(bb), name, up(rb), off)
    ez, ey = forward_bounds(y, z, mag, K, name, up(rb))
    yo, yflat = _out((T, N), pad=pad, shift=shift)
    zo, zflat = _out((T, N), pad=pad, shift=shift) if has_z else (None, None)
    q = ve.new_act8(T, N, block, DEV) if block else None
    if q is not None:
        q.codes.fill_(99)
        q.scales.fill_(7)
    args = dict(bias=None if bb is None else _dev(bb), activation=name,
                residual=None if rb is None else _dev(rb, pad, shift), z=zo, z8=q,
                offsets=None if off is None else torch.from_numpy(off).to(DEV))
    x, w = _dev(xb, pad, shift), _dev(wb, pad, shift)
    ve.linear_forward(x, w, yo, **args)
    inside = ~np.isnan(z).any(1)
    got = _host(yo)
    _within(got[inside], y[inside], ey[inside], "y")
    assert (got[~inside] == 7).all() and _untouched(yflat, yo)
    if has_z:
        from linear_common import rounded
        gz = _host(zo)
        _within(gz[inside], z[inside], rounded(ez, z)[inside], "z")
        assert (gz[~inside] == 7).all() and _untouched(zflat, zo)
    if q is not None:
        codes, scales = q.codes.cpu().numpy(), q.scales.cpu().numpy().astype(np.float64)
        assert (codes[~inside] == 99).all() and (scales[~inside] == 7).all()
        runs = scales.shape[1]
        pad_z = np.zeros((T, runs * block))
        pad_z[:, :N] = np.abs(np.nan_to_num(z))
        pad_e = np.zeros((T, runs * block))
        pad_e[:, :N] = ez
        amax, emax = (v.reshape(T, runs, block).max(-1) for v in (pad_z, pad_e))
        _within(scales[inside], (amax / 127)[inside], (emax / 127 + 2.0 ** -23 * (amax + emax) / 127 + 2.0 ** -149)[inside],
                "scales")
        # a code is within half a step (and the rounding of v * inv, 2^-15 of a step) of the value it saves
        step = np.repeat(scales, block, 1)[:, :N]
        _within((codes * step)[inside], z[inside], (step * (0.5 + 2.0 ** -14) + 2 * np.repeat(emax, block, 1)[:, :N])[inside],
                "codes")
    return x, w, yo, args, inside


@pytest.mark.parametrize("case", FORWARD, ids=lambda c: "-".join(map(str, c)))
def test_forward(case):
    print(f"[gpu] forward {case}", flush=True)
    _forward_case(*case)


# every form of the product where it applies, and split contractions
@pytest.mark.parametrize("path,split", [(1, 1), (2, 0), (2, 1), (3, 0), (3, 1)])
@pytest.mark.parametrize("case", [
    (200, 1096, 392, None, "gelu", True, True, True, 64, 0, 0),
    (65, 2056, 136, None, "silu", True, False, False, 128, 0, 0),
    (333, 264, 392, 7, "none", True, True, True, 32, 0, 0),
    (530, 64, 520, None, "none", False, False, False, 0, 0, 0),
], ids=lambda c: "-".join(map(str, c)))
def test_forward_forms(case, path, split):
    ve = _ve()
    print(f"[gpu] forward {case} path {path} split {split}", flush=True)
    with ve.options(linear_path=path, linear_split=split):
        _forward_case(*case)


@pytest.mark.parametrize("case", [
    (1, 8, 8, None, "none", True, True, True, 0, 0, 0),
    (2, 2056, 24, None, "gelu", True, False, False, 0, 8, 8),
    (3, 1000, 1031, None, "silu", True, True, True, 0, 0, 0),
    (4, 4616, 37, None, "relu", True, True, False, 0, 0, 0),
    (7, 4104, 4100, None, "gelu_tanh", True, True, False, 0, 0, 0),
    (1, 8192, 4099, None, "none", True, False, False, 0, 0, 0),
    (8, 136, 16400, None, "none", False, False, False, 0, 0, 0),
    (5, 99, 75, None, "silu", True, True, True, 0, 3, 1),       # not 16-byte rows: another form takes it
], ids=lambda c: "-".join(map(str, c)))
def test_forward_of_few_tokens(case):
    ve = _ve()
    print(f"[gpu] forward of few tokens {case}", flush=True)
    with ve.options(linear_path=4):
        _forward_case(*case)


def test_forward_residual_in_place_and_repeat():
    import torch
    ve = _ve()
    x, w, y, args, _ = _forward_case(130, 264, 392, None, "silu", True, True, False, 0, 0, 0)
    again = args["residual"].clone()
    ve.linear_forward(x, w, again, **{**args, "residual": again})
    torch.cuda.synchronize()
    assert torch.equal(again, y)


def test_forward_of_no_tokens_and_no_group_rows():
    import torch
    ve = _ve()
    w = _dev(_bits((3, 16, 8), 1))
    e = torch.empty(0, 8, dtype=torch.bfloat16, device=DEV)
    ve.linear_forward(e, w, torch.empty(0, 16, dtype=torch.bfloat16, device=DEV),
                      offsets=torch.zeros(4, dtype=torch.int64, device=DEV))
    y, flat = _out((9, 16))
    ve.linear_forward(_dev(_bits((9, 8), 2)), w, y, offsets=torch.full((4,), 4, dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()
    assert bool((flat == 7).all())


def test_infinities_and_nan_pass_through():
    import torch
    ve = _ve()
    K, N = 64, 40
    xb, wb = _bits((5, K), 1), _bits((N, K), 2)
    xb[1, 3], xb[2, 5] = 0x7FC0, 0x7F80
    x, w = _dev(xb), _dev(wb)
    for name in linear.ACTS:
        y = torch.empty(5, N, dtype=torch.bfloat16, device=DEV)
        ve.linear_forward(x, w, y, activation=name)
        ref, z, mag = linear.forward(_up(xb), _up(wb), None, name)
        _, ey = forward_bounds(ref, z, mag, K, name)
        got = _host(y)
        for r in (0, 3, 4):
            _within(got[r], ref[r], ey[r], name)
        assert np.isnan(got[1]).all()
        assert np.array_equal(got[2], ref[2])            # +-inf, or the limit 0


# ---------------------------------------------------------------------------
# backward

BACKWARD = [
    # T, K, N, groups, act, saved block (0: bf16), bias, dx_add, fp32, accumulate, pad, shift
    (1, 1, 1, None, "none", 0, True, False, True, False, 0, 0),
    (1, 64, 40, None, "silu", 0, True, True, False, False, 0, 0),
    (3, 7, 5, None, "gelu", 32, True, True, False, True, 0, 0),
    (77, 200, 136, None, "none", 0, True, False, True, False, 0, 0),
    (64, 128, 256, None, "relu", 64, False, False, False, False, 0, 0),
    (130, 264, 520, None, "gelu_tanh", 128, True, True, False, True, 0, 0),
    (129, 99, 75, None, "silu", 32, True, False, True, True, 1, 3),
    (300, 136, 264, None, "gelu", 0, True, False, False, False, 8, 8),
    (2100, 72, 40, None, "none", 128, True, False, True, False, 0, 0),
    (40, 136, 264, 1, "silu", 64, True, False, False, False, 0, 0),
    (333, 264, 136, 7, "gelu", 0, True, True, False, False, 0, 0),
    (333, 99, 75, 7, "silu", 32, True, False, True, True, 3, 1),
    (700, 64, 136, 70, "relu", 0, True, False, False, True, 0, 0),
    (200, 80, 72, 130, "none", 0, True, False, False, False, 8, 0),
]


def _backward_case(T, K, N, E, name, block, has_bias, has_add, fp32, accumulate, pad, shift, seed=0):
    import torch
    ve = _ve()
    off = None if E is None else group_offsets(T, E, seed + E, first=2 if T > 20 else 0, spare=3 if T > 20 else 0)
    wshape, bshape = ((N, K), (N,)) if E is None else ((E, N, K), (E, N))
    dyb, wb = _bits((T, N), seed + 1, 1e-3), _bits(wshape, seed + 2, K ** -0.5)
    xb, zb = _bits((T, K), seed + 3), _bits((T, N), seed + 4, 1.5)
    ab = _bits((T, K), seed + 5, 1e-3) if has_add else None
    grad = "float32" if fp32 else "bfloat16"
    x, z = _dev(xb, pad, shift), _dev(zb, pad, shift)
    if block:
        saved = []
        for t in (x, z):
            q = ve.new_act8(*t.shape, block, DEV)
            ve.act8_pack(t, q)
            back = torch.empty(*t.shape, dtype=torch.bfloat16, device=DEV)
            ve.act8_unpack(q, back)
            saved.append((q, back))
        (x, rx), (z, rz) = saved
    else:
        rx, rz = x, z
    if name == "none":
        z = None
    dx, dxf = _out((T, K), pad=pad, shift=shift)
    dw, dwf = _out(wshape, grad, pad, shift)
    db, dbf = _out(bshape, grad) if has_bias else (None, None)
    before = None
    if accumulate:
        hw = torch.from_numpy(np.random.default_rng(seed + 6).standard_normal(wshape) * 1e-3).to(dw.dtype)
        hb = torch.from_numpy(np.random.default_rng(seed + 7).standard_normal(bshape) * 1e-3).to(dw.dtype)
        dw.copy_(hw)
        if has_bias:
            db.copy_(hb)
        before = (hw.double().numpy(), hb.double().numpy())
    xv, zv = _host(rx), _host(rz)
    dy, w = _dev(dyb, pad, shift), _dev(wb, pad, shift)
    args = dict(x=x, z=z, activation=name, dx=dx, dx_add=None if ab is None else _dev(ab, pad, shift), dw=dw, dbias=db,
                accumulate=accumulate, offsets=None if off is None else torch.from_numpy(off).to(DEV))
    ve.linear_backward(dy, w, **args)
    av = None if ab is None else _up(ab)
    ref = linear.backward(_up(dyb), _up(wb), xv, zv, name, av, off)
    bound = backward_bounds(ref, _up(dyb), _up(wb), xv, name, off, fp32, av, before)
    inside = ~np.isnan(ref["dx"]).any(1)
    got = _host(dx)
    _within(got[inside], ref["dx"][inside], bound["dx"][inside], "dx")
    assert (got[~inside] == 7).all() and _untouched(dxf, dx)
    _within(_host(dw), ref["dw"] + (before[0] if before else 0), bound["dw"], "dw")
    assert _untouched(dwf, dw)
    if has_bias:
        _within(_host(db), ref["dbias"] + (before[1] if before else 0), bound["dbias"], "dbias")
        assert _untouched(dbf, db)
    return dy, w, args, (rx, rz)


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    print(f"[gpu] backward {case}", flush=True)
    _backward_case(*case)


@pytest.mark.parametrize("path,split", [(1, 1), (2, 0), (2, 1), (3, 0), (3, 1)])
@pytest.mark.parametrize("case", [
    (1100, 136, 264, None, "silu", 64, True, True, False, True, 0, 0),
    (130, 264, 1096, None, "none", 0, True, False, True, False, 0, 0),
    (333, 264, 392, 7, "gelu", 128, True, True, False, False, 0, 0),
], ids=lambda c: "-".join(map(str, c)))
def test_backward_forms(case, path, split):
    ve = _ve()
    print(f"[gpu] backward {case} path {path} split {split}", flush=True)
    with ve.options(linear_path=path, linear_split=split):
        _backward_case(*case)


def test_backward_from_8_bits_equals_from_restored():
    import torch
    ve = _ve()
    for case in ((130, 264, 520, None, "gelu", 64, True, False, False, False, 0, 0),
                 (333, 264, 392, 7, "silu", 128, True, False, True, False, 0, 0)):
        dy, w, args, (rx, rz) = _backward_case(*case)
        got = {k: args[k].clone() for k in ("dx", "dw", "dbias")}
        ve.linear_backward(dy, w, **{**args, "x": rx, "z": rz})
        torch.cuda.synchronize()
        for k, v in got.items():
            assert torch.equal(v, args[k]), k


def test_backward_outputs_are_optional():
    import torch
    ve = _ve()
    dy, w, args, _ = _backward_case(130, 264, 392, None, "silu", 0, True, False, True, False, 0, 0)
    want = {k: args[k].clone() for k in ("dx", "dw", "dbias")}
    for k in want:
        only = {**args, "dx": None, "dw": None, "dbias": None}
        only[k] = torch.full_like(want[k], 7)
        if k != "dw":
            only["x"] = None
        ve.linear_backward(dy, w, **only)
        torch.cuda.synchronize()
        assert torch.equal(only[k], want[k]), k


def test_gradients_are_difference_quotients():
    """<gradient, direction> against the oracle's loss at x +- h, w +- h, b +- h."""
    import torch
    ve = _ve()
    T, K, N, E, h = 90, 72, 56, 3, 1e-4
    off = np.array([0, 31, 31, 90])
    rng = np.random.default_rng(5)
    xb, wb, bb, dyb = _bits((T, K), 1), _bits((E, N, K), 2, K ** -0.5), _bits((E, N), 3), _bits((T, N), 4, 0.1)
    x, w, b, dy = _up(xb), _up(wb), _up(bb), _up(dyb)
    for name in linear.ACTS:
        _, z, _ = linear.forward(x, w, b, name, None, off)
        zb = f64_to_bf16_bits(z)
        dx, dw, db = (torch.empty(s, dtype=t, device=DEV) for s, t in (((T, K), torch.bfloat16),
                      ((E, N, K), torch.float32), ((E, N), torch.float32)))
        ve.linear_backward(_dev(dyb), _dev(wb), x=_dev(xb), z=_dev(zb) if name != "none" else None, activation=name, dx=dx,
                           dw=dw, dbias=db, offsets=torch.from_numpy(off).to(DEV))
        loss = lambda xx, ww, bb_: (linear.forward(xx, ww, bb_, name, None, off)[0] * dy).sum()  # noqa: E731
        ref = linear.backward(dy, w, x, z, name, None, off)
        for got, key, at in ((dx, "dx", 0), (dw, "dw", 1), (db, "dbias", 2)):
            d = rng.standard_normal(ref[key].shape)
            args = [x, w, b]
            plus, minus = list(args), list(args)
            plus[at], minus[at] = args[at] + h * d, args[at] - h * d
            want = (loss(*plus) - loss(*minus)) / (2 * h)
            # z, dz and the result are each rounded to bf16 (2^-8, slopes change by at most |z| 2^-8); relu's
            # kink flips nothing at these sizes
            scale = np.linalg.norm(ref[key]) * np.sqrt(d.size) * 2.0 ** -8 * 3
            assert abs((_host(got) * d).sum() - want) <= scale, (name, key)
        if E > 1:
            assert not dw[1].any() and not db[1].any()


def test_empty_groups_keep_theirs_with_accumulate():
    import torch
    ve = _ve()
    off = torch.tensor([0, 0, 5, 5], dtype=torch.int64, device=DEV)
    dy, w, x = _dev(_bits((5, 24), 1)), _dev(_bits((3, 24, 16), 2)), _dev(_bits((5, 16), 3))
    dw, db = torch.full((3, 24, 16), 3.0, device=DEV), torch.full((3, 24), 3.0, device=DEV)
    ve.linear_backward(dy, w, x=x, dw=dw, dbias=db, accumulate=True, offsets=off)
    torch.cuda.synchronize()
    assert bool((dw[[0, 2]] == 3).all()) and bool((db[[0, 2]] == 3).all()) and not bool((dw[1] == 3).all())
    ve.linear_backward(dy, w, x=x, dw=dw, dbias=db, offsets=off)
    torch.cuda.synchronize()
    assert not dw[[0, 2]].any() and not db[[0, 2]].any()
    e = torch.empty(0, 24, dtype=torch.bfloat16, device=DEV)
    dw.fill_(3), db.fill_(3)
    ve.linear_backward(e, w, x=torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), dw=dw, dbias=db,
                       offsets=torch.zeros(4, dtype=torch.int64, device=DEV))
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_bad_offsets_stay_inside_the_buffers():
    """Offsets that decrease or leave [0, tokens] give some values, but only inside the outputs."""
    import torch
    ve = _ve()
    x, w, dy = _dev(_bits((50, 32), 1)), _dev(_bits((4, 40, 32), 2)), _dev(_bits((50, 40), 3))
    for off in ([-5, 20, 10, 60, 1 << 40], [50, 0, 50, 0, 50], [0, 0, 0, 0, 0]):
        o = torch.tensor(off, dtype=torch.int64, device=DEV)
        y, yf = _out((50, 40), pad=8, shift=8)
        dx, dxf = _out((50, 32), pad=8, shift=8)
        dw, dwf = _out((4, 40, 32), "float32", 8, 8)
        ve.linear_forward(x, w, y, offsets=o)
        ve.linear_backward(dy, w, x=x, dx=dx, dw=dw, dbias=torch.empty(4, 40, device=DEV), offsets=o)
        torch.cuda.synchronize()
        assert _untouched(yf, y) and _untouched(dxf, dx) and _untouched(dwf, dw)


def test_refusals_of_the_binding():
    import torch
    ve = _ve()
    x, w, y = _dev(_bits((4, 8), 1)), _dev(_bits((16, 8), 2)), torch.zeros(4, 16, dtype=torch.bfloat16, device=DEV)
    for kw, match in ((dict(bias=y[0].half()), "bf16"), (dict(bias=y[0, :8]), "shape"), (dict(z8=ve.new_act8(4, 8, 32, DEV)), "shape"),
                      (dict(residual=y.t()), "shape"), (dict(z8=ve.Act8(y, y, 33)), "block"),
                      (dict(workspace=torch.zeros(0, dtype=torch.float32, device=DEV)), "workspace"),
                      (dict(offsets=torch.zeros(2, dtype=torch.int64)), "contiguous on"),
                      (dict(stream=torch.cuda.Stream(DEV), activation="swish"), "unknown activation")):
        with pytest.raises(ValueError, match=match):
            ve.linear_forward(x, w, y, **kw)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        ve.linear_forward(x, w, torch.zeros(16, 4, dtype=torch.bfloat16, device=DEV).t())
    with pytest.raises(ValueError, match="needs z"):
        ve.linear_backward(y, w, x=x, dw=torch.zeros_like(w), activation="silu")
    with pytest.raises(ValueError, match="needs x"):
        ve.linear_backward(y, w, dw=torch.zeros_like(w))
    with pytest.raises(ValueError, match="both bf16 or both fp32"):
        ve.linear_backward(y, w, x=x, dw=torch.zeros_like(w), dbias=torch.zeros(16, device=DEV))
    torch.cuda.synchronize()
    assert not y.any()


# ---------------------------------------------------------------------------
# sizes and strides whose offsets pass 32 bits

def test_offsets_beyond_32_bits():
    """Outputs of more than 2^31 elements (4.6 GB), checked on sampled rows;
    the last rows lie past 2^32 bytes."""
    import torch
    ve = _ve()
    T, K, N = 70001, 64, 32776
    assert T * N > 2 ** 31
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device=DEV).to(torch.bfloat16)
    y = torch.zeros(T, N, dtype=torch.bfloat16, device=DEV)
    q = ve.new_act8(T, N, 128, DEV)
    for kw in ({}, {"z8": q}):
        y.zero_()
        ve.linear_forward(x, w, y, **kw)
        rows = [0, 1, 255, 256, 33000, 65519, 65520, 65536, 69999, 70000]
        xs, ws = _host(x[rows]), _host(w)
        ref, z, mag = linear.forward(xs, ws)
        _, ey = forward_bounds(ref, z, mag, K, "none")
        _within(_host(y[rows]), ref, ey, "y")
    back = torch.empty_like(y)
    ve.act8_unpack(q, back)
    torch.cuda.synchronize()
    got, want = back[rows].float(), y[rows].float()
    step = q.scales[rows].repeat_interleave(128, 1)[:, :N]
    assert bool(((got - want).abs() <= 0.5 * step * 1.001 + 2.0 ** -7 * want.abs()).all())
    p = ve.new_act8(T, N, 128, DEV)
    ve.act8_pack(y, p)
    torch.cuda.synchronize()
    codes, scales = linear.pack(_host(y[rows]).astype(np.float32), 128)
    assert np.array_equal(p.codes[rows].cpu().numpy(), codes) and np.array_equal(p.scales[rows].cpu().numpy(), scales)
    # dz w and dz^T x over the same rows: the contraction of 70,001 tokens against a float64 product of a column sample
    dx, dw = torch.empty_like(x), torch.empty(N, K, dtype=torch.float32, device=DEV)
    db = torch.empty(N, dtype=torch.float32, device=DEV)
    y.mul_(2.0 ** -6)
    ve.linear_backward(y, w, x=x, dx=dx, dw=dw, dbias=db)
    cols = [0, 7, 127, 128, 16384, 32768, 32775]
    dy, xv = _host(y[:, cols]), _host(x)
    from linear_common import gamma
    _within(_host(dw[cols]), dy.T @ xv, gamma(T + 34) * (np.abs(dy).T @ np.abs(xv)) + 2.0 ** -126, "dw")
    _within(_host(db[cols]), dy.sum(0), gamma(T + 8) * np.abs(dy).sum(0) + 2.0 ** -126, "dbias")
    dyr = _host(y[rows])
    r = dyr @ ws
    _within(_host(dx[rows]), r, 2.0 ** -8 * np.abs(r) + 1.01 * gamma(N + 2) * (np.abs(dyr) @ np.abs(ws)) + 2.0 ** -126, "dx")


@pytest.mark.parametrize("ld", [2 ** 21, 2 ** 21 + 8])
def test_long_leading_dimensions(ld):
    """Rows 2^21 elements apart (the direct loads' limit) and just beyond it."""
    import torch
    ve = _ve()
    T, K, N = 40, 64, 72
    xb, wb, dyb = _bits((T, K), 1), _bits((N, K), 2), _bits((T, N), 3)
    x, y, dy, dx = (torch.zeros(T, ld, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    w, dw = (torch.zeros(N, ld, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    x[:, :K], w[:, :K], dy[:, :N] = _dev(xb), _dev(wb), _dev(dyb)
    ve.linear_forward(x[:, :K], w[:, :K], y[:, :N], activation="silu", residual=dy[:, :N])
    ve.linear_backward(dy[:, :N], w[:, :K], x=x[:, :K], dx=dx[:, :K], dx_add=x[:, :K], dw=dw[:, :K])
    ref, z, mag = linear.forward(_up(xb), _up(wb), None, "silu", _up(dyb))
    _within(_host(y[:, :N]), ref, forward_bounds(ref, z, mag, K, "silu", _up(dyb))[1], "y")
    r = linear.backward(_up(dyb), _up(wb), _up(xb), None, "none", _up(xb))
    b = backward_bounds(r, _up(dyb), _up(wb), _up(xb), "none", None, False, _up(xb))
    _within(_host(dx[:, :K]), r["dx"], b["dx"], "dx")
    _within(_host(dw[:, :K]), r["dw"], b["dw"], "dw")
    assert not y[:, N:].any() and not dx[:, K:].any() and not dw[:, K:].any()


# ---------------------------------------------------------------------------
# streams, graphs, and the operators together

def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own (allocated) scratch."""
    import torch
    ve = _ve()
    dy, w, args, _ = _backward_case(1100, 136, 264, None, "silu", 64, True, True, False, False, 0, 0)
    want = {k: args[k].clone() for k in ("dx", "dw", "dbias")}
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    outs = [{k: torch.full_like(v, 7) for k, v in want.items()} for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o in zip(streams, outs):
            ve.linear_backward(dy, w, **{**args, **o}, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for k, v in want.items():
            assert torch.equal(o[k], v), k


def test_short_workspace_is_refused():
    import torch
    ve = _ve()
    dy, w, args, _ = _backward_case(130, 264, 392, None, "silu", 0, True, False, True, False, 0, 0)
    need = ve.linear_backward_workspace(dy, w, **args)
    before = args["dx"].clone()
    for ws in (torch.empty(need - 256, dtype=torch.uint8, device=DEV), torch.empty(need + 256, dtype=torch.uint8, device=DEV)[16:]):
        args["dx"].fill_(5)
        with pytest.raises(ve.VeError, match="workspace"):
            ve.linear_backward(dy, w, workspace=ws, **args)
        torch.cuda.synchronize()
        assert bool((args["dx"] == 5).all())
    args["dx"].copy_(before)


def test_other_stream_and_captured_graph():
    import torch
    ve = _ve()
    fx, fw, fy, fargs, _ = _forward_case(65, 2056, 136, None, "silu", True, False, False, 64, 0, 0)
    dy, w, args, _ = _backward_case(1100, 136, 264, None, "silu", 64, True, True, False, False, 0, 0)
    want = [fy.clone(), fargs["z8"].codes.clone()] + [args[k].clone() for k in ("dx", "dw", "dbias")]

    def outputs():
        return [fy, fargs["z8"].codes] + [args[k] for k in ("dx", "dw", "dbias")]

    def clear():
        for t in outputs():
            t.fill_(1)

    def both(**kw):
        ve.linear_forward(fx, fw, fy, **fargs, **kw)
        ve.linear_backward(dy, w, **args, **kw)

    s = torch.cuda.Stream(DEV)
    for stream in (s, s.cuda_stream):
        clear()
        s.wait_stream(torch.cuda.current_stream())
        both(stream=stream)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(), want))
    nf = ve.linear_forward_workspace(fx, fw, fy, **fargs)
    nb = ve.linear_backward_workspace(dy, w, **args)
    assert nf > 0 and nb > 0
    fws, bws = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in (nf, nb))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ve.linear_forward(fx, fw, fy, workspace=fws, **fargs)
        ve.linear_backward(dy, w, workspace=bws, **args)
    for _ in range(3):
        clear()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(), want))
        both()                                             # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(), want))


def test_layer_gradients_into_a_bucket_and_step():
    """Two layers forward and backward from 8-bit activations, dw and dbias
    straight into the DBuffer bucket (views at the planned offsets), the
    mean over two micro-batches by the group scale, then the shard step; the
    bucket against the oracle's gradients, and the step's gradient slice
    against the bucket."""
    import torch
    ve = _ve()
    T, H, I, E = 96, 64, 136, 3
    shapes = [[E * I, H, 1, H], [E * I, 1, 8, 1], [H, I, 1, I], [H, 1, 8, 1]]    # experts' up + bias, down + bias
    specs, S, _ = ve.plan_layout(np.array(shapes), 2, 16)
    plan = ve.Plan(specs, 2, S, device=0)
    bucket = torch.full((2 * S,), 9.0, dtype=torch.bfloat16, device=DEV)
    plan.group_op(-1, ve.GROUP_ZERO, 0.0, ve.group_table(plan, -1, [bucket]))
    view = [bucket[o:o + r * c] for r, c, _, _, o in specs.tolist()]
    gw1, gb1, gw2, gb2 = view[0].view(E, I, H), view[1].view(E, I), view[2].view(H, I), view[3]
    w1, b1, w2, b2 = (_bits(s, 10 + i, 0.1) for i, s in enumerate(((E, I, H), (E, I), (H, I), (H,))))
    off = np.array([0, 40, 40, T])
    doff = torch.from_numpy(off).to(DEV)
    up = _up
    want = [np.zeros((E, I, H)), np.zeros((E, I)), np.zeros((H, I)), np.zeros(H)]
    tol = [np.zeros_like(v) for v in want]
    for mb in range(2):
        xb, dyb = _bits((T, H), 20 + mb), _bits((T, H), 30 + mb, 0.1)
        x, dy = _dev(xb), _dev(dyb)
        h, y = (torch.empty(T, n, dtype=torch.bfloat16, device=DEV) for n in (I, H))
        z8, x8, h8 = ve.new_act8(T, I, 32, DEV), ve.new_act8(T, H, 32, DEV), ve.new_act8(T, I, 32, DEV)
        ve.linear_forward(x, _dev(w1), h, bias=_dev(b1), activation="gelu", z8=z8, offsets=doff)
        ve.linear_forward(h, _dev(w2), y, bias=_dev(b2), residual=x)
        ve.act8_pack(x, x8)
        ve.act8_pack(h, h8)
        dh, dx = torch.empty_like(h), torch.empty_like(x)
        ve.linear_backward(dy, _dev(w2), x=h8, dx=dh, dw=gw2, dbias=gb2, accumulate=True)
        ve.linear_backward(dh, _dev(w1), x=x8, z=z8, activation="gelu", dx=dx, dx_add=dy, dw=gw1, dbias=gb1,
                           accumulate=True, offsets=doff)
        # the layers' values against the oracle, each from the inputs the GPU gave it
        y1, zz, mag = linear.forward(up(xb), up(w1), up(b1), "gelu", None, off)
        _within(_host(h), y1, forward_bounds(y1, zz, mag, H, "gelu")[1], "h")
        hv = _host(h)
        y2, zz, mag = linear.forward(hv, up(w2), up(b2), "none", up(xb))
        _within(_host(y), y2, forward_bounds(y2, zz, mag, I, "none", up(xb))[1], "y")
        rest = []
        for q, n in ((h8, I), (x8, H), (z8, I)):
            t = torch.empty(T, n, dtype=torch.bfloat16, device=DEV)
            ve.act8_unpack(q, t)
            rest.append(_host(t))
        r2 = linear.backward(up(dyb), up(w2), rest[0], None, "none")
        bd2 = backward_bounds(r2, up(dyb), up(w2), rest[0], "none", None, False, before=(want[2], want[3]))
        _within(_host(dh), r2["dx"], bd2["dx"], "dh")
        r1 = linear.backward(_host(dh), up(w1), rest[1], rest[2], "gelu", up(dyb), off)
        bd1 = backward_bounds(r1, _host(dh), up(w1), rest[1], "gelu", off, False, up(dyb), before=(want[0], want[1]))
        _within(_host(dx), r1["dx"], bd1["dx"], "dx")
        got = [_host(g) for g in (gw1, gb1, gw2, gb2)]
        for i, (g, r, b) in enumerate(zip(got, (r1["dw"], r1["dbias"], r2["dw"], r2["dbias"]),
                                          (bd1["dw"], bd1["dbias"], bd2["dw"], bd2["dbias"]))):
            _within(g, want[i] + r, b, f"bucket {i}")
            want[i] = g                                    # the next micro-batch adds to what is there
    mask = torch.ones(2 * S, dtype=torch.bool, device=DEV)
    for r, c, _, _, o in specs.tolist():
        mask[o:o + r * c] = False
    assert not bucket[mask].any()                          # padding stays 0
    plan.group_op(-1, ve.GROUP_SCALE, 0.5, ve.group_table(plan, -1, [bucket]))
    grads = ve.grad_pointer_table([v.contiguous() for v in view], DEV)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
    for rank in range(2):
        master = torch.randn(S, device=DEV)
        st = ve.new_state(plan, rank, grads, master.clone())
        plan.step(rank, ve.state_table(plan, rank, [st]), hp, 1)
        torch.cuda.synchronize()
        assert torch.equal(st["grad_shard"].view(torch.bfloat16), bucket[rank * S:(rank + 1) * S])
        moved = (st["master"] - master).abs()
        assert bool((moved[bucket[rank * S:(rank + 1) * S] != 0] > 0).all())
    plan.close()


# ---------------------------------------------------------------------------
# rows that are not whole 16 bytes: operands laid out anew in the workspace

LAID_OUT_FORWARD = [
    (65, 2053, 139, None, "silu", True, False, False, 128, 0, 0),
    (200, 1091, 397, None, "gelu", True, True, True, 64, 3, 1),
    (300, 136, 520, None, "none", False, True, False, 0, 4, 4),      # whole rows at addresses that are not
    (130, 1, 257, None, "relu", False, False, False, 0, 0, 0),
    (333, 99, 75, 7, "silu", True, True, True, 32, 3, 1),
    (700, 63, 135, 70, "none", True, False, False, 0, 0, 0),
]
LAID_OUT_BACKWARD = [
    (1100, 135, 263, None, "silu", 64, True, True, False, True, 0, 0),
    (130, 263, 1091, None, "none", 0, True, False, True, False, 1, 3),
    (129, 264, 75, None, "gelu", 128, True, False, True, False, 0, 0),  # out_features alone is odd
    (129, 99, 136, None, "none", 0, True, True, False, False, 0, 0),    # in_features alone is odd
    (300, 136, 264, None, "relu", 0, True, False, False, False, 4, 4),
    (333, 261, 397, 7, "gelu", 128, True, True, False, False, 0, 0),
    (700, 63, 135, 70, "none", 0, True, False, False, True, 2, 1),
]


def _poison(bytes_):
    """A workspace whose every bf16 and fp32 is NaN."""
    import torch
    return torch.full((bytes_ or 1,), 255, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("path,split", [(2, 0), (2, 1), (3, 0), (3, 1)])
@pytest.mark.parametrize("case", LAID_OUT_FORWARD, ids=lambda c: "-".join(map(str, c)))
def test_forward_of_rows_laid_out_anew(case, path, split):
    import torch
    ve = _ve()
    print(f"[gpu] forward {case} path {path} split {split}", flush=True)
    with ve.options(linear_path=path, linear_split=split):
        x, w, y, args, _ = _forward_case(*case)
        want = y.clone()
        y.fill_(7)
        need = ve.linear_forward_workspace(x, w, y, **args)
        assert need > 0
        ve.linear_forward(x, w, y, workspace=_poison(need), **args)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("path,split", [(2, 0), (2, 1), (3, 0), (3, 1)])
@pytest.mark.parametrize("case", LAID_OUT_BACKWARD, ids=lambda c: "-".join(map(str, c)))
def test_backward_of_rows_laid_out_anew(case, path, split):
    import torch
    ve = _ve()
    print(f"[gpu] backward {case} path {path} split {split}", flush=True)
    with ve.options(linear_path=path, linear_split=split):
        dy, w, args, _ = _backward_case(*case)
        args["accumulate"] = False
        outs = ("dx", "dw", "dbias")
        ve.linear_backward(dy, w, **args)
        want = {k: args[k].clone() for k in outs}
        for k in outs:
            args[k].fill_(7)
        need = ve.linear_backward_workspace(dy, w, **args)
        assert need > 0
        ve.linear_backward(dy, w, workspace=_poison(need), **args)
        torch.cuda.synchronize()
        inside = slice(None)
        if args["offsets"] is not None:
            off = args["offsets"].tolist()
            inside = slice(off[0], off[-1])
        assert torch.equal(args["dx"][inside], want["dx"][inside])
        for k in ("dw", "dbias"):
            assert torch.equal(args[k], want[k]), k


@pytest.mark.parametrize("case", [
    (2051, 1037, 1203, None, "gelu", 64, True, False, False, False, 0, 0),
    (130, 263, 521, None, "silu", 32, True, False, False, False, 0, 0),
    (33, 1037, 1203, None, "silu", 32, True, False, False, False, 0, 0),
    (700, 101, 136, None, "relu", 64, True, False, True, False, 0, 0),
    (2100, 263, 75, None, "gelu", 64, True, False, True, False, 0, 0),   # long contraction, few tiles
    (333, 261, 397, 7, "silu", 128, True, False, True, False, 0, 0),
], ids=lambda c: "-".join(map(str, c)))
def test_odd_backward_from_8_bits_equals_from_restored(case):
    import torch
    ve = _ve()
    dy, w, args, (rx, rz) = _backward_case(*case)
    got = {k: args[k].clone() for k in ("dx", "dw", "dbias")}
    ve.linear_backward(dy, w, **{**args, "x": rx, "z": rz})
    torch.cuda.synchronize()
    for k, v in got.items():
        assert torch.equal(v, args[k]), k


def test_rows_laid_out_anew_in_a_captured_graph():
    import torch
    ve = _ve()
    with ve.options(linear_path=2):
        x, w, y, fargs, _ = _forward_case(200, 1091, 397, None, "gelu", True, False, False, 0, 3, 1)
        dy, w2, args, _ = _backward_case(130, 263, 1091, None, "none", 0, True, False, True, False, 1, 3)
        outs = [y] + [args[k] for k in ("dx", "dw", "dbias")]
        want = [t.clone() for t in outs]
        fws, bws = _poison(ve.linear_forward_workspace(x, w, y, **fargs)), _poison(ve.linear_backward_workspace(dy, w2, **args))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ve.linear_forward(x, w, y, workspace=fws, **fargs)
            ve.linear_backward(dy, w2, workspace=bws, **args)
        for _ in range(3):
            for t in outs:
                t.fill_(1)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            ve.linear_forward(x, w, y, **fargs)
            ve.linear_backward(dy, w2, **args)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
        # what the operands hold at the replay counts, not at the capture
        x.mul_(2)
        ve.linear_forward(x, w, y, **fargs)
        torch.cuda.synchronize()
        twice = y.clone()
        y.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, twice) and not torch.equal(y, want[0])
