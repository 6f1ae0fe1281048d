"""Refusals of the entry points on matrices in 8-bit floating point, on the C
ABI without a GPU: every call here is rejected before anything reaches a
device, or has nothing to launch."""

from __future__ import annotations

import ctypes as C

import pytest

import ragged_shard_optimizer_amd as ve
from oracle import fp8

P = 1 << 24  # never dereferenced; buffers lie 16 MiB apart
BAD, OK, UNSUP = ve.VE_ERR_INVALID_ARG, ve.VE_OK, ve.VE_ERR_UNSUPPORTED


def _q(at, rows, cols, block=1, fmt=0, **kw):
    whole, n = -(-cols // 16) * 16, -(-rows // block)
    q = ve._Fp8(at * P, whole, at * P + P // 2, -(-n // 4) * 4, fmt, block)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


@pytest.mark.parametrize("rows,groups", [(0, 1), (1, 1), (1, 5), (127, 1), (129, 2), (1000, 64), (5, 100)])
def test_columns(rows, groups):
    assert ve.fp8_columns(rows, groups) == (fp8.columns(rows, groups) if rows else 0)
    assert ve.fp8_columns(-3, 1) == ve.fp8_columns(3, 0) == 0


SPOILED = [dict(codes=None), dict(scales=None), dict(format=2), dict(format=-1), dict(block_rows=0), dict(block_rows=64),
           dict(ld_codes=8), dict(ld_codes=120), dict(codes=9 * P + 8), dict(scales=9 * P + 2), dict(ld_scales=2), dict(ld_scales=301)]


def _pack(**kw):
    a = ve._Fp8Pack(rows=300, cols=100, groups=1, x=P, ldx=100, out=_q(2, 300, 100), out_t=_q(3, 100, 384))
    for k, v in kw.items():
        setattr(a, k, v)
    return ve.lib().ve_fp8_pack(C.byref(a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=0, x=None), OK), (dict(out=ve._Fp8(), out_t=ve._Fp8()), OK),
    (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(groups=0), BAD), (dict(groups=2), BAD), (dict(x=None), BAD),
    (dict(ldx=99), BAD), (dict(activation=5), BAD), (dict(activation=4), BAD), (dict(activation=4, z=4 * P, ldz=99), BAD),
    (dict(out_t=_q(3, 100, 300)), BAD), (dict(out_t=_q(3, 100, 384, fmt=1)), BAD), (dict(out=_q(1, 300, 100)), BAD),
    (dict(out_t=_q(2, 100, 384)), BAD), (dict(offsets=2 * P), BAD), (dict(offsets=4 * P, groups=65537), BAD),
    (dict(rows=1 << 31), UNSUP), (dict(rows=1 << 30, cols=1 << 20, ldx=1 << 20, out=_q(2, 1 << 30, 1 << 20), out_t=ve._Fp8()), UNSUP),
] + [(dict(out=_q(2, 300, 100, **s)), BAD) for s in SPOILED[1:]] + [(dict(out_t=_q(3, 100, 384, **s)), BAD) for s in SPOILED[1:-1]])
def test_pack_checks(kw, rc):
    assert _pack(**kw) == rc
    assert rc == OK or ve.lib().ve_last_error()


@pytest.mark.parametrize("kw,rc", [
    (dict(out=ve._Fp8(), out_t=ve._Fp8()), OK), (dict(rows=0), BAD), (dict(w=None), BAD), (dict(ldw=99), BAD),
    (dict(out=_q(2, 300, 100, 1)), BAD), (dict(out_t=_q(2, 100, 300, 128)), BAD), (dict(groups=2, w_group=29999), BAD),
    (dict(groups=2, w_group=30000), BAD), (dict(groups=2, w_group=30000, out_codes_group=300 * 112, out_scales_group=2), BAD),
    (dict(groups=2, w_group=30000, out_codes_group=300 * 112 + 8, out_scales_group=4), BAD),
    (dict(out_t=_q(3, 100, 300, 128, fmt=1)), BAD), (dict(cols=1 << 31), UNSUP),
])
def test_pack_weight_checks(kw, rc):
    a = ve._Fp8PackWeight(rows=300, cols=100, groups=1, w=P, ldw=100, out=_q(2, 300, 100, 128), out_t=_q(3, 100, 300, 128))
    for k, v in kw.items():
        setattr(a, k, v)
    assert ve.lib().ve_fp8_pack_weight(C.byref(a), None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=0, x=None), OK), (dict(x=None), BAD), (dict(ldx=99), BAD), (dict(rows=-1), BAD), (dict(groups=0), BAD),
    (dict(x=2 * P + 16), BAD), (dict(groups=2, in_codes_group=300 * 112, in_scales_group=300, x_group=29999), BAD),
    (dict(groups=2, in_codes_group=300 * 112 - 16, in_scales_group=300, x_group=30000), BAD),
    (dict(groups=2, in_codes_group=300 * 112, in_scales_group=296, x_group=30000), BAD), (dict(rows=1 << 31), UNSUP),
] + [(dict(in_=_q(2, 300, 100, **s)), BAD) for s in SPOILED])
def test_unpack_checks(kw, rc):
    a = ve._Fp8Unpack(rows=300, cols=100, groups=1, in_=_q(2, 300, 100), x=P, ldx=100)
    for k, v in kw.items():
        setattr(a, k, v)
    assert ve.lib().ve_fp8_unpack(C.byref(a), None) == rc
    assert ve.lib().ve_fp8_unpack(None, None) == BAD


def _fwd(**kw):
    a = ve._Fp8Forward(tokens=300, in_features=100, out_features=200, groups=1, activation=0, x=_q(1, 300, 100),
                       w=_q(2, 200, 100, 128), y=3 * P, ldy=200)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), (dict(tokens=0, x=ve._Fp8(), y=None), OK), (dict(x=_q(1, 300, 100, fmt=1)), OK),
    (dict(tokens=-1), BAD), (dict(in_features=0), BAD), (dict(out_features=0), BAD), (dict(groups=0), BAD), (dict(groups=2), BAD),
    (dict(activation=5), BAD), (dict(y=None), BAD), (dict(ldy=199), BAD), (dict(residual=4 * P, ldr=199), BAD),
    (dict(z=4 * P, ldz=199), BAD), (dict(w=_q(2, 200, 100, 1)), BAD), (dict(w=_q(2, 200, 100, 128, fmt=1)), BAD),
    (dict(x=_q(1, 300, 100, 128)), BAD), (dict(groups=3, offsets=5 * P, w_codes_group=200 * 112 - 16, w_scales_group=4), BAD),
    (dict(groups=3, offsets=5 * P, w_codes_group=200 * 112, w_scales_group=4), OK),
    (dict(groups=3, offsets=5 * P, w_codes_group=200 * 112, w_scales_group=4, bias=6 * P, bias_group=199), BAD),
    (dict(tokens=1 << 31), UNSUP), (dict(x=_q(1, 300, 100, ld_codes=(1 << 22) + 16)), UNSUP),
] + [(dict(x=_q(1, 300, 100, **s)), BAD) for s in SPOILED] + [(dict(w=_q(2, 200, 100, 128, **s)), BAD) for s in SPOILED[:-2]])
def test_forward_checks(kw, rc):
    n = C.c_int64(-1)
    L = ve.lib()
    assert L.ve_fp8_linear_forward_workspace(C.byref(_fwd(**kw)), C.byref(n)) == rc
    if rc != OK:
        assert L.ve_last_error()
        assert L.ve_fp8_linear_forward(C.byref(_fwd(**kw)), None, 0, None) == rc
    else:
        assert n.value >= 0


@pytest.mark.parametrize("kw", [dict(y=P), dict(y=2 * P), dict(y=P + P // 2), dict(z=3 * P, ldz=200), dict(residual=3 * P, ldr=208),
                                dict(offsets=3 * P), dict(bias=3 * P + 2)])
def test_forward_refuses_overlaps(kw):
    a = _fwd(**kw)
    n = C.c_int64()
    assert ve.lib().ve_fp8_linear_forward_workspace(C.byref(a), C.byref(n)) == OK
    assert ve.lib().ve_fp8_linear_forward(C.byref(a), 64 * P, n.value, None) == BAD


def _bwd(**kw):
    a = ve._Fp8Backward(tokens=300, in_features=100, out_features=200, groups=1, dy=_q(1, 300, 200), w_t=_q(2, 100, 200, 128),
                        dx=3 * P, lddx=100, dy_t=_q(4, 200, 384), x_t=_q(5, 100, 384), dw=6 * P, lddw=100)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,rc", [
    ({}, OK), (dict(dx=None, dy=ve._Fp8(), w_t=ve._Fp8()), OK), (dict(dw=None, dy_t=ve._Fp8(), x_t=ve._Fp8()), OK),
    (dict(dy=_q(1, 300, 200, fmt=1), dy_t=_q(4, 200, 384, fmt=1)), OK), (dict(tokens=0, dy_t=ve._Fp8(), x_t=ve._Fp8(), dy=ve._Fp8()), OK),
    (dict(dy=ve._Fp8()), BAD), (dict(w_t=ve._Fp8()), BAD), (dict(dy_t=ve._Fp8()), BAD), (dict(x_t=ve._Fp8()), BAD),
    (dict(w_t=_q(2, 100, 200, 128, fmt=1)), BAD), (dict(x_t=_q(5, 100, 384, fmt=1)), BAD), (dict(w_t=_q(2, 100, 200, 1)), BAD),
    (dict(x_t=_q(5, 100, 300)), BAD), (dict(dy_t=_q(4, 200, 368)), BAD), (dict(lddx=99), BAD), (dict(lddw=99), BAD),
    (dict(dx_add=7 * P, ld_add=99), BAD), (dict(groups=2), BAD),
    (dict(groups=2, offsets=8 * P, w_codes_group=100 * 208, w_scales_group=8, dw_group=19999, dy_t=_q(4, 200, 512),
          x_t=_q(5, 100, 512)), BAD),
    (dict(groups=2, offsets=8 * P, w_codes_group=100 * 208, w_scales_group=8, dw_group=20000, dy_t=_q(4, 200, 384),
          x_t=_q(5, 100, 384)), BAD),
    (dict(groups=2, offsets=8 * P, w_codes_group=100 * 208, w_scales_group=8, dw_group=20000, dy_t=_q(4, 200, 512),
          x_t=_q(5, 100, 512)), OK),
    (dict(tokens=1 << 31), UNSUP), (dict(dy=_q(1, 300, 200, ld_codes=(1 << 22) + 16)), UNSUP),
])
def test_backward_checks(kw, rc):
    n = C.c_int64(-1)
    L = ve.lib()
    assert L.ve_fp8_linear_backward_workspace(C.byref(_bwd(**kw)), C.byref(n)) == rc
    if rc != OK:
        assert L.ve_last_error()
        assert L.ve_fp8_linear_backward(C.byref(_bwd(**kw)), None, 0, None) == rc


@pytest.mark.parametrize("kw", [dict(dx=P), dict(dw=4 * P), dict(dx=6 * P), dict(dx_add=3 * P, ld_add=104), dict(dw=5 * P + P // 2)])
def test_backward_refuses_overlaps(kw):
    a = _bwd(**kw)
    n = C.c_int64()
    assert ve.lib().ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == OK
    assert ve.lib().ve_fp8_linear_backward(C.byref(a), 64 * P, n.value, None) == BAD


def test_null_records():
    L = ve.lib()
    n = C.c_int64()
    assert L.ve_fp8_pack(None, None) == L.ve_fp8_pack_weight(None, None) == BAD
    assert L.ve_fp8_linear_forward(None, None, 0, None) == L.ve_fp8_linear_backward(None, None, 0, None) == BAD
    assert L.ve_fp8_linear_forward_workspace(C.byref(_fwd()), None) == BAD
    assert L.ve_fp8_linear_backward_workspace(None, C.byref(n)) == BAD


def test_binding_refusals():
    import torch
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    q, w = ve.new_fp8(4, 16, device="cpu"), ve.new_fp8(8, 16, 128, device="cpu")
    assert q.codes.shape == (4, 16) and q.scales.shape == (1, 4) and w.scales.shape == (1, 1) and w.scales.stride(0) == 4
    for call in (lambda: ve.fp8_pack(x, q), lambda: ve.fp8_pack(x, q, activation="silu"), lambda: ve.fp8_pack(x, q, activation="elu"),
                 lambda: ve.fp8_unpack(q, x), lambda: ve.fp8_pack_weight(x[0], q),
                 lambda: ve.fp8_linear_forward(q, w, torch.zeros(4, 8, dtype=torch.bfloat16)),
                 lambda: ve.fp8_linear_backward(dx=x), lambda: ve.fp8_linear_backward(dw=x),
                 lambda: ve.Fp8(x, q.scales)._fill(4, 16, "q", x.device), lambda: ve.Fp8(q.codes, q.scales, 2)._fill(4, 16, "q", x.device)):
        with pytest.raises(ValueError):
            call()
