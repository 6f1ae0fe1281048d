"""A layer of experts in training, from a router's choice to every gradient,
with its products in 8-bit floating point: each step's output against the fp64
oracle of that step, computed from what the step before left on the device,
within that operator's own bounds."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import expert, fp8, linear
from fp8_common import DEV, cut, cut_rows, forward_bounds, host
from linear_common import TINY, U, gamma, rounded

pytestmark = pytest.mark.gpu


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], bound[bad][:4])


def _values(q):
    c, e = host(q)
    fmt = "e4m3" if "e4m3" in str(q.codes.dtype) else "e5m2"
    if c.ndim == 2:
        return fp8.unpack(c, e, q.block_rows, fmt)
    return np.stack([fp8.unpack(a, b, q.block_rows, fmt) for a, b in zip(c, e)])


@pytest.mark.parametrize("T,k,E,H,F,dtype", [(96, 4, 12, 264, 392, "e4m3"), (300, 2, 8, 136, 520, "e5m2")])
def test_layer_of_experts(T, k, E, H, F, dtype):
    import torch

    import ragged_shard_optimizer_amd as ve
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    R, C = T * k, fp8.columns(T * k, E)
    x, dy = rand(T, H).bfloat16(), (1e-2 * rand(T, H)).bfloat16()
    w1, w2 = (rand(E, F, H) * H ** -0.5).bfloat16(), (rand(E, H, F) * F ** -0.5).bfloat16()
    b1 = (0.1 * rand(E, F)).bfloat16()
    top = torch.topk(rand(T, E), k, dim=1)
    weights, ids = torch.softmax(top.values, 1), top.indices
    ids[3, 0], ids[5] = -1, -1                             # a slot, and a token, over capacity
    # forward
    off, pos = torch.empty(E + 1, dtype=torch.int64, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    ve.expert_sort(ids, off, pos)
    xs, x8, xt = bf(R, H), ve.new_fp8(R, H, device=DEV), ve.new_fp8(H, C, device=DEV)
    ve.expert_gather(x, pos, x8)
    ve.expert_gather(x, pos, xs)
    ve.fp8_pack(xs, None, xt, offsets=off)
    q1, q1t, q2, q2t = (ve.new_fp8(n, m, 128, groups=E, device=DEV) for n, m in ((F, H), (H, F), (H, F), (F, H)))
    ve.fp8_pack_weight(w1, q1, q1t)
    ve.fp8_pack_weight(w2, q2, q2t)
    z, h, o = bf(R, F), bf(R, F), bf(R, H)
    ve.fp8_linear_forward(x8, q1, h, bias=b1, activation="silu", z=z, offsets=off)
    h8, ht = ve.new_fp8(R, F, device=DEV), ve.new_fp8(F, C, device=DEV)
    ve.fp8_pack(h, h8, ht, offsets=off)
    ve.fp8_linear_forward(h8, q2, o, offsets=off)
    y = bf(T, H)
    ve.expert_combine(o, pos, y, weights=weights, residual=x)
    # backward
    do, dweights = bf(R, H), torch.empty(T, k, device=DEV)
    ve.expert_combine_backward(dy, pos, rows=o, weights=weights, drows=do, dweights=dweights)
    do8, dot = ve.new_fp8(R, H, format=dtype, device=DEV), ve.new_fp8(H, C, format=dtype, device=DEV)
    ve.fp8_pack(do, do8, dot, offsets=off)
    dh, dw2 = bf(R, F), torch.empty(E, H, F, device=DEV)
    ve.fp8_linear_backward(dy=do8, w_t=q2t, dx=dh, dy_t=dot, x_t=ht, dw=dw2, offsets=off)
    dz8, dzt = ve.new_fp8(R, F, format=dtype, device=DEV), ve.new_fp8(F, C, format=dtype, device=DEV)
    ve.fp8_pack(dh, dz8, dzt, z=z, activation="silu", offsets=off)
    dxs, dw1 = bf(R, H), bf(E, F, H)
    ve.fp8_linear_backward(dy=dz8, w_t=q1t, dx=dxs, dy_t=dzt, x_t=xt, dw=dw1, offsets=off)
    db1 = torch.empty(E, F, device=DEV)
    ve.linear_backward(dh, w1, z=z, activation="silu", dbias=db1, offsets=off)
    dx = bf(T, H)
    ve.expert_combine(dxs, pos, dx, residual=dy)

    # every step from the one before
    roff, rpos, order = expert.sort(ids.cpu().numpy(), E)
    assert np.array_equal(off.cpu().numpy(), roff) and np.array_equal(pos.cpu().numpy(), rpos)
    n = len(order)
    assert np.array_equal(_host(xs)[:n], _host(x)[order // k])
    vx, v1, v1t, v2, v2t, vh = (_values(q) for q in (x8, q1, q1t, q2, q2t, h8))
    assert np.array_equal(vx[:n], fp8.unpack(*fp8.pack(_host(xs)))[:n])
    assert np.array_equal(v1, np.swapaxes(v1t, 1, 2)) and np.array_equal(v2, np.swapaxes(v2t, 1, 2))
    ry, rz, mag = linear.forward(vx, v1, _host(b1), "silu", None, roff)
    bz, bh = forward_bounds(ry, rz, mag, cut_rows(vx, v1, roff), H, "silu")
    _within(_host(z)[:n], rz[:n], bz[:n], "z")
    _within(_host(h)[:n], ry[:n], bh[:n], "h")
    assert np.array_equal(vh[:n], fp8.unpack(*fp8.pack(_host(h)))[:n])
    ro, rz2, mag = linear.forward(vh, v2, offsets=roff)
    _within(_host(o)[:n], ro[:n], forward_bounds(ro, rz2, mag, cut_rows(vh, v2, roff), F, "none")[1][:n], "o")
    wn = weights.double().cpu().numpy()
    r, mag = expert.combine(_host(o), rpos, wn, _host(x))
    _within(_host(y), r, rounded(gamma(k + 1) * mag, r), "y")
    rdo, rdw, mag = expert.combine_backward(_host(dy), rpos, _host(o), wn)
    _within(_host(do)[:n], rdo[:n], rounded(U * np.abs(rdo), rdo)[:n], "do")
    _within(_host(dweights), rdw, gamma(H + 8) * mag + TINY, "dweights")
    used = sum(-(-int(b - a) // 128) * 128 for a, b in zip(roff, roff[1:]))
    for dyq, dyt, wt, xtq, got, dwt, wide in ((do8, dot, v2t, ht, dh, dw2, True), (dz8, dzt, v1t, xt, dxs, dw1, False)):
        vd, vdt, vxt = _values(dyq), _values(dyt)[:, :used], _values(xtq)[:, :used]
        W = np.swapaxes(wt, 1, 2)
        ref = linear.backward(vd, W, offsets=roff)["dx"]
        mag = linear.backward(np.abs(vd), np.abs(W), offsets=roff)["dx"]
        bound = rounded(gamma(vd.shape[1] + 2) * mag + cut_rows(vd, wt, roff) + TINY, ref)
        _within(_host(got)[:n], ref[:n], bound[:n], "dx of a product")
        ref, mag = fp8.weight_gradient(vdt, vxt, roff, R)
        bound = gamma(R + 130) * mag + TINY
        if not wide:
            at = 0
            for e, (a, b) in enumerate(zip(roff, roff[1:])):
                end = at + -(-int(b - a) // 128) * 128
                bound[e] += cut(vdt[:, at:end], vxt[:, at:end])
                at = end
        _within(_host(dwt), ref, bound if wide else rounded(bound, ref), "dw")
    r, mag = expert.combine(_host(dxs), rpos, None, _host(dy))
    _within(_host(dx), r, rounded(gamma(k + 1) * mag, r), "dx")
    assert np.array_equal(_host(dx)[5], _host(dy)[5])      # a token without experts passes its gradient on
