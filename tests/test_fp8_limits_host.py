"""Sizes at the limits of products on matrices in 8-bit floating point, on the C
ABI without a GPU: what the header allows is taken, what lies past it refused."""

from __future__ import annotations

import ctypes as C

import pytest

import ragged_shard_optimizer_amd as ve

P = 1 << 36  # never dereferenced; buffers lie 64 GiB apart
BAD, OK, UNSUP = ve.VE_ERR_INVALID_ARG, ve.VE_OK, ve.VE_ERR_UNSUPPORTED
PITCH, COLUMNS = 1 << 22, (1 << 24) - 128  # of x, w, dy and w_t; of dy_t and x_t


def _q(at, rows, cols, block=1, ld=None):
    return ve._Fp8(at * P, -(-cols // 16) * 16 if ld is None else ld, at * P + P // 2, -(-rows // (4 * block)) * 4, 0, block)


def _dw(tokens, groups, N=40, K=24, wide=0, ld=None):
    cols = ve.fp8_columns(tokens, groups)
    a = ve._Fp8Backward(tokens=tokens, in_features=K, out_features=N, groups=groups, offsets=P if groups > 1 else None,
                        dy_t=_q(2, N, cols, ld=ld), x_t=_q(3, K, cols), dw=4 * P, lddw=K, dw_group=N * K, grad_fp32=wide)
    n = C.c_int64(-1)
    return ve.lib().ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)), n.value


@pytest.mark.parametrize("wide", [0, 1])
@pytest.mark.parametrize("path", [0, 2, 3])
@pytest.mark.parametrize("tokens,groups,rc", [
    (40000, 40000, OK), (65536, 65536, OK), (1 << 20, 65536, OK),
    (COLUMNS, 1, OK), (COLUMNS + 1, 1, UNSUP), (COLUMNS - 127 * 65536, 65536, OK), (COLUMNS - 127 * 65536 + 128, 65536, UNSUP)])
def test_columns_of_a_weight_gradient(tokens, groups, rc, path, wide):
    assert ve.fp8_columns(tokens, groups) <= COLUMNS or rc != OK
    with ve.options(linear_path=path):
        got, need = _dw(tokens, groups, wide=wide)
    assert got == rc, ve.lib().ve_last_error()
    assert rc != OK or need >= 0
    assert rc == OK or b"2^24" in ve.lib().ve_last_error()


def test_rows_further_apart_than_they_are_long():
    assert _dw(300, 1, ld=(1 << 24) - 16)[0] == OK
    assert _dw(300, 1, ld=1 << 24)[0] == UNSUP


@pytest.mark.parametrize("ld,rc", [(PITCH, OK), (PITCH + 16, UNSUP)])
def test_rows_of_the_other_operands(ld, rc):
    L, n = ve.lib(), C.c_int64(-1)
    for which in ("x", "w"):
        a = ve._Fp8Forward(tokens=300, in_features=100, out_features=200, groups=1, activation=0, y=3 * P, ldy=200,
                           x=_q(1, 300, 100, ld=ld if which == "x" else None), w=_q(2, 200, 100, 128, ld if which == "w" else None))
        assert L.ve_fp8_linear_forward_workspace(C.byref(a), C.byref(n)) == rc
        a = ve._Fp8Backward(tokens=300, in_features=200, out_features=100, groups=1, dx=3 * P, lddx=200,
                            dy=_q(1, 300, 100, ld=ld if which == "x" else None), w_t=_q(2, 200, 100, 128, ld if which == "w" else None))
        assert L.ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == rc


def test_one_gradient_is_not_refused_for_the_other_ones_size():
    """16 million tokens of 8192 features are too many tiles of dx, 65,536 weights
    of 1024 x 1024 too many of dw."""
    L, n, T, E = ve.lib(), C.c_int64(-1), 1 << 20, 65536
    a = ve._Fp8Backward(tokens=T * 15, in_features=8192, out_features=8192, groups=1, dy_t=_q(2, 8192, T * 15), x_t=_q(3, 8192, T * 15),
                        dw=4 * P, lddw=8192)
    assert L.ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == OK
    a.dx, a.lddx, a.dy, a.w_t = 5 * P, 8192, _q(6, T * 15, 8192), _q(7, 8192, 8192, 128)
    assert L.ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == UNSUP
    a = ve._Fp8Backward(tokens=300, in_features=1024, out_features=1024, groups=E, offsets=P, dx=5 * P, lddx=1024,
                        dy=_q(6, 300, 1024), w_t=_q(7, 1024, 1024, 128), w_codes_group=1 << 20, w_scales_group=64)
    assert L.ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == OK
    cols = ve.fp8_columns(300, E)
    a.dw, a.lddw, a.dw_group, a.dy_t, a.x_t = 4 * P, 1024, 1 << 20, _q(2, 1024, cols), _q(3, 1024, cols)
    assert L.ve_fp8_linear_backward_workspace(C.byref(a), C.byref(n)) == UNSUP
