"""Refusals of the linear layer's and the 8-bit code's entry points, on the
C ABI without a GPU: every call here is rejected before anything reaches a
device, or has nothing to launch."""

from __future__ import annotations

import ctypes as C

import pytest

import ragged_shard_optimizer_amd as ve

P = 4096  # never dereferenced
BAD, OK, UNSUP = ve.VE_ERR_INVALID_ARG, ve.VE_OK, ve.VE_ERR_UNSUPPORTED


def _fwd(**kw):
    a = ve._LinearForward(tokens=8, in_features=16, out_features=24, groups=1, activation=0, x=P, ldx=16, w=P, ldw=16,
                          y=2 * P, ldy=24)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _bwd(**kw):
    a = ve._LinearBackward(tokens=8, in_features=16, out_features=24, groups=1, activation=0, dy=P, lddy=24, w=P,
                           ldw=16, x=P, ldx=16, dx=2 * P, lddx=16, dw=P, lddw=16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _q(a, fn):
    n = C.c_int64(-1)
    rc = fn(C.byref(a), C.byref(n))
    return rc, n.value


@pytest.mark.parametrize("kw,rc", [
    ({}, OK),
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(y=P), BAD),
    (dict(tokens=0, x=None, y=None), OK),
    (dict(tokens=-1), BAD), (dict(in_features=0), BAD), (dict(out_features=0), BAD),
    (dict(tokens=1 << 31), UNSUP),
    (dict(tokens=(1 << 31) - 1, out_features=(1 << 31) - 1, ldy=1 << 31), UNSUP),
    (dict(ldx=15), BAD), (dict(ldw=15), BAD), (dict(ldy=23), BAD), (dict(residual=P, ldr=23), BAD),
    (dict(z=P, ldz=23), BAD),
    (dict(groups=0), BAD), (dict(groups=2), BAD), (dict(groups=65537, offsets=P, w_group=400), BAD),
    (dict(groups=2, offsets=P, w_group=383), BAD), (dict(groups=2, offsets=P, w_group=384), OK),
    (dict(groups=2, offsets=P, w_group=384, bias=P, bias_group=23), BAD),
    (dict(activation=-1), BAD), (dict(activation=5), BAD),
    (dict(z8=ve._Act8(P, 24, None, 1, 32)), BAD), (dict(z8=ve._Act8(P, 24, P, 1, 16)), BAD),
    (dict(z8=ve._Act8(P, 23, P, 1, 32)), BAD), (dict(z8=ve._Act8(P, 24, P, 0, 32)), BAD),
    (dict(z8=ve._Act8(P, 24, P, 1, 32)), OK),
])
def test_forward_checks(kw, rc):
    got, need = _q(_fwd(**kw), ve.lib().ve_linear_forward_workspace)
    assert got == rc
    if rc != OK:
        assert ve.lib().ve_last_error()
        assert ve.lib().ve_linear_forward(C.byref(_fwd(**kw)), None, 0, None) == rc
    else:
        assert need >= 0


@pytest.mark.parametrize("kw,rc", [
    ({}, OK),
    (dict(dy=None), BAD), (dict(w=None), BAD), (dict(w=None, dx=None), OK), (dict(x=None), BAD),
    (dict(x=None, dw=None), OK), (dict(x8=ve._Act8(P, 16, P, 1, 32)), BAD),
    (dict(x=None, x8=ve._Act8(P, 16, P, 1, 32)), OK), (dict(x=None, x8=ve._Act8(P, 16, P, 1, 48)), BAD),
    (dict(activation=4), BAD), (dict(activation=4, z=P, ldz=24), OK), (dict(activation=4, z=P, ldz=23), BAD),
    (dict(activation=4, z=P, ldz=24, z8=ve._Act8(P, 24, P, 1, 32)), BAD),
    (dict(activation=4, z8=ve._Act8(P, 24, P, 1, 32)), OK),
    (dict(dx=P), BAD), (dict(lddy=23), BAD), (dict(ldw=15), BAD), (dict(lddx=15), BAD), (dict(lddw=15), BAD), (dict(ldx=15), BAD),
    (dict(dx_add=P, ld_add=15), BAD),
    (dict(groups=3, offsets=P, w_group=384, dw_group=383), BAD),
    (dict(groups=3, offsets=P, w_group=383, dw_group=384), BAD),
    (dict(groups=3, offsets=P, w_group=384, dw_group=384, dbias=P, dbias_group=23), BAD),
    (dict(groups=3, offsets=P, w_group=384, dw_group=384), OK),
    (dict(activation=7, z=P, ldz=24), BAD),
])
def test_backward_checks(kw, rc):
    got, need = _q(_bwd(**kw), ve.lib().ve_linear_backward_workspace)
    assert got == rc
    if rc != OK:
        assert ve.lib().ve_last_error()
        assert ve.lib().ve_linear_backward(C.byref(_bwd(**kw)), None, 0, None) == rc
    else:
        assert need >= 0


def test_null_records_and_workspace():
    L = ve.lib()
    n = C.c_int64()
    assert L.ve_linear_forward(None, None, 0, None) == BAD
    assert L.ve_linear_backward(None, None, 0, None) == BAD
    assert L.ve_linear_forward_workspace(C.byref(_fwd()), None) == BAD
    assert L.ve_linear_backward_workspace(None, C.byref(n)) == BAD
    a = _bwd(activation=4, z=P, ldz=24)       # dz lives in the workspace
    rc, need = _q(a, L.ve_linear_backward_workspace)
    assert rc == OK and need >= 8 * 24 * 2
    assert L.ve_linear_backward(C.byref(a), None, 0, None) == BAD
    assert L.ve_linear_backward(C.byref(a), P, need - 1, None) == BAD
    assert b"workspace" in L.ve_last_error()
    assert L.ve_linear_backward(C.byref(a), P + 16, need, None) == BAD
    assert b"aligned" in L.ve_last_error()
    assert L.ve_linear_forward(C.byref(_fwd(tokens=0, x=None, y=None)), None, 0, None) == OK


def test_act8_checks():
    L = ve.lib()
    q = ve._Act8(P, 100, P, 4, 32)
    for f in (lambda rows, cols, x, ld, q: L.ve_act8_pack(x, ld, rows, cols, q, None),
              lambda rows, cols, x, ld, q: L.ve_act8_unpack(q, rows, cols, x, ld, None)):
        assert f(0, 100, None, 100, C.byref(q)) == OK
        assert f(4, 100, P, 100, None) == BAD
        assert f(4, 100, None, 100, C.byref(q)) == BAD
        assert f(-1, 100, P, 100, C.byref(q)) == BAD
        assert f(4, 0, P, 100, C.byref(q)) == BAD
        assert f(4, 100, P, 99, C.byref(q)) == BAD
        assert f(4, 101, P, 101, C.byref(q)) == BAD           # codes rows too short
        assert f(4, 100, P, 100, C.byref(ve._Act8(P, 100, P, 3, 32))) == BAD
        assert f(4, 100, P, 100, C.byref(ve._Act8(P, 100, P, 4, 33))) == BAD
        assert f(4, 100, P, 100, C.byref(ve._Act8(None, 100, P, 4, 32))) == BAD
        assert f(1 << 40, 100, P, 100, C.byref(q)) == UNSUP
    assert L.ve_last_error()


def test_binding_refuses_host_tensors_and_bad_names():
    import torch
    x, w, y = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 8), (16, 8), (4, 16)))
    with pytest.raises(ValueError, match="device tensor"):
        ve.linear_forward(x, w, y)
    with pytest.raises(ValueError, match="unknown activation"):
        ve.linear_forward(x, w, y, activation="tanh")
    with pytest.raises(ValueError, match="device tensor"):
        ve.act8_pack(x, ve.new_act8(4, 8, device="cpu"))
    with pytest.raises(ValueError, match="1-D int64"):
        ve.linear_forward(x, w, y, offsets=torch.zeros(2, dtype=torch.int32))


def test_workspace_of_rows_laid_out_anew():
    L = ve.lib()
    big = dict(tokens=4096, in_features=4097, out_features=4099, ldx=4097, ldw=4097, ldy=4099)
    rc, need = _q(_fwd(**big), L.ve_linear_forward_workspace)
    assert rc == OK and need >= (4096 + 4099) * 4104 * 2
    whole = dict(tokens=4096, in_features=4096, out_features=4096, ldx=4096, ldw=4096, ldy=4096)
    rc, need = _q(_fwd(**whole), L.ve_linear_forward_workspace)
    assert rc == OK and need == 0
    with ve.options(linear_path=1):
        rc, need = _q(_fwd(**big), L.ve_linear_forward_workspace)
        assert rc == OK and need == 0
    # an operand too large for one copying launch is read where it lies
    top = (1 << 31) - 1
    rc, need = _q(_fwd(tokens=1, in_features=top, out_features=1 << 20, ldx=top, ldw=top, ldy=1 << 20),
                  L.ve_linear_forward_workspace)
    assert rc == OK and need < 1 << 40


Q = 1 << 40  # the buffers of these records lie far apart, but for the one that is moved


def _apart_fwd(**kw):
    a = ve._LinearForward(tokens=8, in_features=16, out_features=24, groups=2, activation=0, offsets=Q, x=2 * Q, ldx=16,
                          w=3 * Q, ldw=16, w_group=400, y=4 * Q, ldy=24, bias=5 * Q, bias_group=32, residual=6 * Q, ldr=24,
                          z=7 * Q, ldz=24, z8=ve._Act8(8 * Q, 24, 9 * Q, 1, 32))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _apart_bwd(**kw):
    a = ve._LinearBackward(tokens=8, in_features=16, out_features=24, groups=2, activation=4, offsets=Q, dy=2 * Q, lddy=24,
                           w=3 * Q, ldw=16, w_group=400, x=4 * Q, ldx=16, z=5 * Q, ldz=24, dx=6 * Q, lddx=16, dx_add=7 * Q,
                           ld_add=16, dw=8 * Q, lddw=16, dw_group=400, dbias=9 * Q, dbias_group=32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _refused(fn, query, a, names, workspace=10 * Q):
    n = C.c_int64()
    assert query(C.byref(a), C.byref(n)) == OK
    assert fn(C.byref(a), workspace, n.value, None) == BAD
    msg = ve.lib().ve_last_error().decode()
    assert "overlaps" in msg and all(w in msg for w in names), msg


@pytest.mark.parametrize("kw,names", [
    (dict(y=2 * Q + 32), "yx"), (dict(y=3 * Q), "yw"), (dict(y=3 * Q + 800), "yw"), (dict(y=5 * Q + 64), ("y", "bias")),
    (dict(y=6 * Q + 48), ("y", "residual")), (dict(y=6 * Q, ldy=32), ("y", "residual")), (dict(y=Q + 8), ("y", "offsets")),
    (dict(x=4 * Q + 48 * 7), "yx"), (dict(z=4 * Q), "yz"), (dict(z=2 * Q), "zx"),
    (dict(z8=ve._Act8(2 * Q + 1, 24, 9 * Q, 1, 32)), ("codes", "x")), (dict(z8=ve._Act8(8 * Q, 24, 7 * Q, 1, 32)), ("scales", "z")),
    (dict(z8=ve._Act8(8 * Q, 24, 8 * Q + 24, 1, 32)), ("codes", "scales")),
])
def test_forward_outputs_over_other_buffers(kw, names):
    L = ve.lib()
    _refused(L.ve_linear_forward, L.ve_linear_forward_workspace, _apart_fwd(**kw), names)


@pytest.mark.parametrize("kw,names", [
    (dict(dx=4 * Q), ("dx", "x")), (dict(dx=4 * Q + 32), ("dx", "x")), (dict(dx=3 * Q), ("dx", "w")), (dict(dx=5 * Q), ("dx", "z")),
    (dict(dx=2 * Q + 48), ("dx", "dy")), (dict(dx=7 * Q, lddx=24), ("dx", "dx_add")), (dict(dx=7 * Q + 32), ("dx", "dx_add")),
    (dict(dx=8 * Q), ("dx", "dw")), (dict(dw=2 * Q), ("dw", "dy")), (dict(dw=4 * Q), ("dw", "x")), (dict(dw=3 * Q), ("dw", "w")),
    (dict(dbias=2 * Q + 2), ("dbias", "dy")), (dict(dbias=8 * Q + 832), ("dw", "dbias")), (dict(dx=10 * Q), ("dx", "workspace")),
    (dict(x=None, x8=ve._Act8(6 * Q, 16, 11 * Q, 1, 32)), ("dx", "codes")),
    (dict(x=None, x8=ve._Act8(11 * Q, 16, 6 * Q, 1, 32)), ("dx", "scales")),
    (dict(z=None, z8=ve._Act8(8 * Q, 24, 11 * Q, 1, 32)), ("dw", "codes")),
])
def test_backward_outputs_over_other_buffers(kw, names):
    L = ve.lib()
    _refused(L.ve_linear_backward, L.ve_linear_backward_workspace, _apart_bwd(**kw), names)


def test_act8_over_other_buffers():
    L = ve.lib()
    for codes, scales in ((2 * Q, 3 * Q), (2 * Q + 200, 3 * Q), (3 * Q, 2 * Q + 4), (3 * Q, 3 * Q + 100)):
        q = ve._Act8(codes, 100, scales, 4, 32)
        assert L.ve_act8_pack(2 * Q, 100, 4, 100, C.byref(q), None) == BAD
        assert b"overlaps" in L.ve_last_error()
    q = ve._Act8(3 * Q, 100, 4 * Q, 4, 32)
    for x in (3 * Q, 3 * Q + 1, 4 * Q - 200):
        assert L.ve_act8_unpack(C.byref(q), 4, 100, x, 100, None) == BAD
        assert b"overlaps" in L.ve_last_error()
