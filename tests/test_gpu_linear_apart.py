"""GPU: buffers that are interleaved but apart are taken (column slices of one
allocation, a group's gradients between the groups' weights)."""

from __future__ import annotations

import pytest

from test_gpu_linear import DEV, _bits, _dev, _ve

pytestmark = pytest.mark.gpu


def _side_by_side(*tensors):
    """Copies as column slices of one buffer."""
    import torch
    buf = torch.empty(*tensors[0].shape[:-1], sum(t.shape[-1] for t in tensors), dtype=torch.bfloat16, device=DEV)
    out, at = [], 0
    for t in tensors:
        v = buf[..., at:at + t.shape[-1]]
        v.copy_(t)
        out.append(v)
        at += t.shape[-1]
    return out


@pytest.mark.parametrize("K,N", [(64, 136), (99, 75)])
@pytest.mark.parametrize("E", [None, 3])
def test_column_slices_of_one_buffer(K, N, E):
    import torch
    ve = _ve()
    T = 130
    print(f"[gpu] slices {K} {N} {E}", flush=True)
    x, z, dy, add = (_dev(_bits((T, n), i)) for i, n in enumerate((K, N, N, K)))
    w = _dev(_bits((N, K) if E is None else (E, N, K), 9))
    off = None if E is None else torch.tensor([0, 50, 50, T], dtype=torch.int64, device=DEV)
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    ve.linear_forward(x, w, y, activation="silu", residual=dy, offsets=off)
    ve.linear_backward(dy, w, x=x, z=z, activation="silu", dx=dx, dx_add=add, dw=dw, offsets=off)
    xs, zs, dys, adds, ys, dxs = _side_by_side(x, z, dy, add, torch.empty_like(y), torch.empty_like(dx))
    ws, dws = _side_by_side(w, torch.empty_like(w))
    ve.linear_forward(xs, ws, ys, activation="silu", residual=dys, offsets=off)
    ve.linear_backward(dys, ws, x=xs, z=zs, activation="silu", dx=dxs, dx_add=adds, dw=dws, offsets=off)
    torch.cuda.synchronize()
    for got, want in ((xs, x), (zs, z), (dys, dy), (adds, add), (ws, w)):
        assert torch.equal(got, want)                       # the inputs are as they were
    # another alignment may cut the contraction elsewhere: fp32 sums of up to 136 products of at most 3 (sums of
    # magnitudes below 400) within 2 * 136 * 2^-23 * 400 = 0.013 of one another, then one step of bf16
    for got, want in ((ys, y), (dxs, dx), (dws, dw)):
        assert bool(((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -6).all())


def test_gradients_between_the_weights():
    """dw of a group behind the weights of that group, in one allocation."""
    import torch
    ve = _ve()
    T, K, N, E = 96, 64, 40, 3
    x, dy, w = _dev(_bits((T, K), 1)), _dev(_bits((T, N), 2)), _dev(_bits((E, N, K), 3))
    off = torch.tensor([0, 30, 61, T], dtype=torch.int64, device=DEV)
    both = torch.zeros(E, 2, N, K, dtype=torch.bfloat16, device=DEV)
    both[:, 0] = w
    dx, want = torch.empty_like(x), torch.empty_like(w)
    ve.linear_backward(dy, w, x=x, dx=dx, dw=want, offsets=off)
    ve.linear_backward(dy, both[:, 0], x=x, dx=dx, dw=both[:, 1], offsets=off)
    torch.cuda.synchronize()
    assert torch.equal(both[:, 1], want) and torch.equal(both[:, 0], w)


def test_overlap_is_refused_before_anything_runs():
    import torch
    ve = _ve()
    x, dy, w = _dev(_bits((96, 64), 1)), _dev(_bits((96, 64), 2)), _dev(_bits((64, 64), 3))
    held, dw = x.clone(), torch.full_like(w, 7)
    with pytest.raises(ve.VeError, match="dx overlaps x"):
        ve.linear_backward(dy, w, x=x, dx=x, dw=dw)
    torch.cuda.synchronize()
    assert torch.equal(x, held) and bool((dw == 7).all())
    ve.linear_backward(dy, w, dx=x)                         # x is not read: dx may stand there
    want = torch.empty_like(x)
    ve.linear_backward(dy, w, dx=want)
    torch.cuda.synchronize()
    assert torch.equal(x, want)
