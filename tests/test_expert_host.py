"""Refusals of the entry points that sort slots by expert and bring rows there
and back, on the C ABI without a GPU: every call here is rejected before
anything reaches a device, or has nothing to launch."""

from __future__ import annotations

import ctypes as C

import pytest

import ragged_shard_optimizer_amd as ve

P = 1 << 20  # never dereferenced; buffers lie 1 MiB apart
BAD, OK, UNSUP = ve.VE_ERR_INVALID_ARG, ve.VE_OK, ve.VE_ERR_UNSUPPORTED


def _need(tokens, slots, experts):
    n = C.c_int64(-1)
    return ve.lib().ve_expert_sort_workspace(tokens, slots, experts, C.byref(n)), n.value


@pytest.mark.parametrize("tokens,slots,experts,rc", [
    (8, 2, 4, OK), (0, 1, 1, OK), (-1, 1, 1, BAD), (8, 0, 4, BAD), (8, 65, 4, BAD), (8, 2, 0, BAD), (8, 2, 4097, BAD),
    (8, 64, 4096, OK), (1 << 30, 2, 4, UNSUP), ((1 << 30) - 1, 2, 4, OK),
])
def test_sort_sizes(tokens, slots, experts, rc):
    got, need = _need(tokens, slots, experts)
    assert got == rc
    if rc == OK:
        assert 0 <= need <= 256 * 4096 * 4
    else:
        assert ve.lib().ve_last_error()


def test_sort_workspace_is_small():
    assert _need(0, 8, 256) == (OK, 0)
    assert _need(256, 8, 256) == (OK, 0) and _need(257, 8, 256) == (OK, 2 * 256 * 4)
    assert ve.expert_sort_workspace(1 << 20, 8, 256) == 256 * 256 * 4
    assert ve.lib().ve_expert_sort_workspace(8, 2, 4, None) == BAD


def test_sort_checks():
    f = ve.lib().ve_expert_sort
    ok = dict(e=P, ib=8, T=8, k=2, n=4, off=2 * P, pos=3 * P, order=None, ws=None, size=0)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["e"], a["ib"], a["T"], a["k"], a["n"], a["off"], a["pos"], a["order"], a["ws"], a["size"], None)

    for kw in (dict(ib=2), dict(e=None), dict(off=None), dict(pos=None), dict(off=P), dict(pos=P), dict(pos=2 * P),
               dict(order=3 * P), dict(order=P + 8), dict(n=0), dict(k=0), dict(T=-1),
               dict(T=4096, k=8), dict(T=4096, k=8, ws=4 * P, size=16), dict(T=4096, k=8, ws=4 * P + 4, size=1 << 20)):
        assert call(**kw) == BAD, kw
    assert call(T=1 << 31) == UNSUP


def _gather(**kw):
    a = ve._ExpertGather(tokens=8, cols=100, slots=2, position=P, x=2 * P, ldx=100, rows_len=16, rows=3 * P, ld_rows=100)
    for k, v in kw.items():
        setattr(a, k, v)
    return ve.lib().ve_expert_gather(C.byref(a), None)


Q = ve._Fp8(4 * P, 112, 5 * P, 16, 0, 1)


def _q(**kw):
    q = ve._Fp8(4 * P, 112, 5 * P, 16, 0, 1)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


@pytest.mark.parametrize("kw,rc", [
    (dict(tokens=0, position=None, x=None), OK), (dict(rows_len=0), OK),
    (dict(tokens=-1), BAD), (dict(cols=0), BAD), (dict(slots=0), BAD), (dict(slots=65), BAD), (dict(rows_len=-1), BAD),
    (dict(position=None), BAD), (dict(x=None), BAD), (dict(rows=None), BAD), (dict(ldx=99), BAD), (dict(ld_rows=99), BAD),
    (dict(rows8=Q), BAD), (dict(rows=None, rows8=Q, weights=6 * P), BAD), (dict(rows=2 * P), BAD), (dict(rows=P), BAD),
    (dict(x=3 * P + 200), BAD), (dict(weights=3 * P + 2), BAD),
    (dict(rows=None, rows8=_q(format=2)), BAD), (dict(rows=None, rows8=_q(block_rows=128)), BAD),
    (dict(rows=None, rows8=_q(ld_codes=96)), BAD), (dict(rows=None, rows8=_q(ld_codes=104)), BAD),
    (dict(rows=None, rows8=_q(codes=4 * P + 8)), BAD), (dict(rows=None, rows8=_q(scales=5 * P + 2)), BAD),
    (dict(rows=None, rows8=_q(ld_scales=14)), BAD), (dict(rows=None, rows8=_q(ld_scales=18)), BAD),
    (dict(rows=None, rows8=_q(scales=None)), BAD), (dict(rows=None, rows8=_q(scales=4 * P)), BAD),
    (dict(tokens=1 << 30), UNSUP), (dict(cols=1 << 31, ldx=1 << 31, ld_rows=1 << 31), UNSUP),
    (dict(tokens=1 << 29, cols=1 << 20, ldx=1 << 20, ld_rows=1 << 20), UNSUP), (dict(rows_len=1 << 31), UNSUP),
])
def test_gather_checks(kw, rc):
    assert _gather(**kw) == rc
    assert rc == OK or ve.lib().ve_last_error()


@pytest.mark.parametrize("kw,rc", [
    (dict(tokens=0, position=None, y=None), OK),
    (dict(y=None), BAD), (dict(rows=None), BAD), (dict(position=None), BAD), (dict(ldy=99), BAD), (dict(ld_rows=99), BAD),
    (dict(residual=6 * P, ldr=99), BAD), (dict(y=2 * P), BAD), (dict(residual=3 * P, ldr=104), BAD), (dict(slots=0), BAD),
    (dict(weights=3 * P), BAD), (dict(residual=3 * P + 200, ldr=100), BAD), (dict(tokens=1 << 31), UNSUP),
])
def test_combine_checks(kw, rc):
    a = ve._ExpertCombine(tokens=8, cols=100, slots=2, position=P, rows_len=16, rows=2 * P, ld_rows=100, y=3 * P, ldy=100)
    for k, v in kw.items():
        setattr(a, k, v)
    assert ve.lib().ve_expert_combine(C.byref(a), None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(tokens=0, position=None, dy=None), OK), (dict(drows=None, dweights=None), OK),
    (dict(dy=None), BAD), (dict(rows=None), BAD), (dict(position=None), BAD), (dict(lddy=99), BAD), (dict(ld_rows=99), BAD),
    (dict(ld_drows=99), BAD), (dict(drows=2 * P), BAD), (dict(drows=3 * P), BAD), (dict(dweights=4 * P), BAD),
    (dict(dweights=P), BAD), (dict(weights=4 * P), BAD), (dict(weights=5 * P), BAD), (dict(slots=65), BAD),
    (dict(tokens=1 << 31), UNSUP),
])
def test_combine_backward_checks(kw, rc):
    a = ve._ExpertCombineBackward(tokens=8, cols=100, slots=2, position=P, dy=3 * P, lddy=100, rows_len=16, rows=2 * P,
                                  ld_rows=100, drows=4 * P, ld_drows=100, dweights=5 * P)
    for k, v in kw.items():
        setattr(a, k, v)
    assert ve.lib().ve_expert_combine_backward(C.byref(a), None) == rc


def test_null_records():
    L = ve.lib()
    assert L.ve_expert_gather(None, None) == L.ve_expert_combine(None, None) == L.ve_expert_combine_backward(None, None) == BAD


def test_binding_refuses_host_tensors_and_shapes():
    import torch
    t = torch
    ids, off, pos = t.zeros(4, 2, dtype=t.int64), t.zeros(5, dtype=t.int64), t.zeros(4, 2, dtype=t.int32)
    x = t.zeros(4, 16, dtype=t.bfloat16)
    for call in (lambda: ve.expert_sort(ids, off, pos), lambda: ve.expert_sort(ids[0], off, pos),
                 lambda: ve.expert_sort(ids, off[:1], pos), lambda: ve.expert_gather(x, pos, x),
                 lambda: ve.expert_gather(x, pos[:3], x), lambda: ve.expert_combine(x, pos, x),
                 lambda: ve.expert_combine_backward(x, pos, drows=x)):
        with pytest.raises(ValueError):
            call()
