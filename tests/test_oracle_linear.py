"""Pins of the linear layer's fp64 oracle: against torch's autograd in fp64,
against finite differences, and the 8-bit code's rule by hand."""

from __future__ import annotations

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import linear
from linear_common import group_offsets

TORCH = {"none": lambda z: z, "relu": torch.relu, "gelu": F.gelu, "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"),
         "silu": F.silu}


def _case(T, K, N, E, seed):
    rng = np.random.default_rng(seed)
    off = None if E is None else group_offsets(T, E, seed, first=1, spare=2)
    w = rng.standard_normal((N, K) if E is None else (E, N, K))
    b = rng.standard_normal((N,) if E is None else (E, N))
    return rng.standard_normal((T, K)), w, b, rng.standard_normal((T, N)), rng.standard_normal((T, N)), off


@pytest.mark.parametrize("name", linear.ACTS)
@pytest.mark.parametrize("E", [None, 4])
def test_matches_autograd(name, E):
    x, w, b, r, dy, off = _case(23, 7, 5, E, 3)
    y, z, _ = linear.forward(x, w, b, name, r, off)
    got = linear.backward(dy, w, x, np.nan_to_num(z), name, None, off)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    loss = 0.0
    for e, lo, hi in linear.parts(off, 23):
        we, be = (tw, tb) if E is None else (tw[e], tb[e])
        ty = TORCH[name](tx[lo:hi] @ we.t() + be) + torch.tensor(r[lo:hi])
        assert np.allclose(ty.detach().numpy(), y[lo:hi], rtol=1e-12, atol=1e-12)
        loss = loss + (ty * torch.tensor(dy[lo:hi])).sum()
    loss.backward()
    inside = np.zeros(23, bool)
    for _, lo, hi in linear.parts(off, 23):
        inside[lo:hi] = True
    assert np.allclose(tx.grad.numpy()[inside], got["dx"][inside], rtol=1e-9, atol=1e-11)
    assert np.allclose(tw.grad.numpy(), got["dw"], rtol=1e-9, atol=1e-11)
    assert np.allclose(tb.grad.numpy(), got["dbias"], rtol=1e-9, atol=1e-11)


@pytest.mark.parametrize("name", linear.ACTS)
def test_slope_is_the_difference_quotient(name):
    z = np.linspace(-6, 6, 241) + 0.0123  # off relu's kink
    h = 1e-5
    want = (linear.act(name, z + h) - linear.act(name, z - h)) / (2 * h)
    assert np.abs(linear.slope(name, z) - want).max() < 1e-8


@pytest.mark.parametrize("name", linear.ACTS[1:])
def test_values_at_the_ends(name):
    z = np.array([np.inf, -np.inf, 3e38, -3e38, 0.0])
    y, d = linear.act(name, z), linear.slope(name, z)
    assert y[0] == np.inf and y[1] == 0 and y[2] == 3e38 and y[3] == 0 and y[4] == 0
    assert d[0] == 1 and d[1] == 0 and d[2] == 1 and d[3] == 0
    assert np.isnan(linear.act(name, np.array([np.nan]))[0])


def test_pack_rule_by_hand():
    v = np.zeros((4, 40), np.float32)
    v[0, 0], v[0, 1], v[0, 31], v[0, 32] = 2.54, -1.27, 0.015, 127.0
    v[1, 5] = 1e-39                                        # below fp32's normal range
    v[1, 6] = -5e-40
    v[2, 3] = np.inf
    v[3, 39] = np.nan
    c, s = linear.pack(v, 32)
    assert c[0, :2].tolist() == [127, -64] and c[0, 31] == 1 and c[0, 32] == 127 and s[0, 1] == 1.0
    assert c[1, 5] == 127 and c[1, 6] in (-63, -64) and s[1, 0] > 0
    assert np.isnan(s[2, 0]) and not c[2].any() and s[2, 1] == 0
    assert np.isnan(s[3, 1]) and s[3, 0] == 0
    back = linear.unpack(c, s, 32)
    assert np.isnan(back[2, :32]).all() and not back[2, 32:].any()
    rng = np.random.default_rng(0)
    v = rng.standard_normal((9, 100)).astype(np.float32)
    for block in (32, 64, 128):
        c, s = linear.pack(v, block)
        step = np.repeat(s, block, 1)[:, :100]
        assert (np.abs(linear.unpack(c, s, block) - v) <= step * 0.5001).all()
