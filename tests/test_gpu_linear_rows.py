"""GPU: rows that belong to no group are not read where operands are laid out
anew or restored: none of what they hold gets into the workspace, whose rows
for them keep what they held."""

from __future__ import annotations

import numpy as np
import pytest

from test_gpu_linear import DEV, _bits, _dev, _ve

pytestmark = pytest.mark.gpu

MARK = 0x1234  # a bf16 that no other operand holds (5.7e-28)
T, FIRST, LAST = 300, 40, 250


def _offsets():
    import torch
    return torch.tensor([FIRST, 100, 100, LAST], dtype=torch.int64, device=DEV)


def _marked(cols, seed):
    bits = _bits((T, cols), seed)
    bits[:FIRST] = MARK
    bits[LAST:] = MARK
    return _dev(bits)


def _none(workspace):
    import torch
    torch.cuda.synchronize()
    assert workspace.numel() > 0
    return not bool((workspace.view(torch.int16) == MARK).any())


@pytest.mark.parametrize("path", [2, 3])
def test_forward_reads_the_rows_of_groups(path):
    import torch
    ve = _ve()
    x, w = _marked(99, 1), _dev(_bits((3, 75, 99), 2))
    y = torch.full((T, 75), 7.0, dtype=torch.bfloat16, device=DEV)
    with ve.options(linear_path=path):
        ws = torch.zeros(ve.linear_forward_workspace(x, w, y, offsets=_offsets()), dtype=torch.uint8, device=DEV)
        ve.linear_forward(x, w, y, offsets=_offsets(), workspace=ws)
    assert _none(ws)
    assert bool((y[:FIRST] == 7).all()) and bool((y[LAST:] == 7).all())


@pytest.mark.parametrize("path", [2, 3])
@pytest.mark.parametrize("saved", [False, True])
def test_backward_reads_the_rows_of_groups(path, saved):
    import torch
    ve = _ve()
    dy, x, w = _marked(75, 1), _marked(99, 2), _dev(_bits((3, 75, 99), 3))
    if saved:
        q = ve.new_act8(T, 99, 32, DEV)
        ve.act8_pack(x, q)
        for rows in (slice(0, FIRST), slice(LAST, T)):
            q.codes[rows] = 1
            q.scales[rows] = float(torch.tensor([MARK], dtype=torch.int16).view(torch.bfloat16))
    dx, dw = torch.full((T, 99), 7.0, dtype=torch.bfloat16, device=DEV), torch.empty_like(w)
    args = dict(x=q if saved else x, dx=dx, dw=dw, offsets=_offsets())
    with ve.options(linear_path=path):
        ws = torch.zeros(ve.linear_backward_workspace(dy, w, **args), dtype=torch.uint8, device=DEV)
        ve.linear_backward(dy, w, workspace=ws, **args)
    assert _none(ws)
    assert bool((dx[:FIRST] == 7).all()) and bool((dx[LAST:] == 7).all())
