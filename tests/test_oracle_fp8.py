"""Pins of the 8-bit floating point oracle: the formats' values against torch's
float8 types, codes against a search over all values, exponents by hand."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import expert, fp8

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_values_are_the_formats(fmt):
    want = torch.arange(256, dtype=torch.uint8).view(TORCH[fmt]).double().numpy()
    got = fp8.values(fmt)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.nanmax(got[np.isfinite(got)]) == fp8.MAX[fmt]


@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_codes_are_the_nearest_even(fmt):
    v = fp8.values(fmt)
    pos = v[:128][np.isfinite(v[:128])]                       # ascending
    rng = np.random.default_rng(0)
    mid = (pos[1:] + pos[:-1]) / 2
    y = np.concatenate([pos, mid, mid * (1 + 1e-9), mid * (1 - 1e-9), rng.uniform(0, fp8.MAX[fmt], 1000),
                        np.exp(rng.uniform(-12, 6, 1000)).clip(max=fp8.MAX[fmt])])
    y = np.concatenate([y, -y])
    d = np.abs(np.abs(y)[:, None] - pos[None])
    best = d.min(1)
    want = [min(np.flatnonzero(row == b), key=lambda c: c & 1) for row, b in zip(d, best)]
    got = fp8.encode(y, fmt)
    assert np.array_equal(got & 127, np.array(want)) and np.array_equal(got >> 7, np.signbit(y))


def test_codes_of_non_finite_values():
    y = np.array([np.inf, -np.inf, np.nan])
    assert fp8.encode(y, "e4m3").tolist()[:2] == [0x7F, 0xFF] and fp8.encode(y, "e4m3")[2] & 127 == 0x7F
    assert fp8.encode(y, "e5m2").tolist()[:2] == [0x7C, 0xFC] and fp8.encode(y, "e5m2")[2] & 127 == 0x7F


def test_exponents_by_hand():
    a = np.array([0.0, 448.0, 448.0001, 224.0, 1.0, 2.0 ** -133, 1.75, 1.7501])
    assert fp8.exponents(a, "e4m3").tolist() == [0, 127, 128, 126, 119, 0, 119, 120]
    assert fp8.exponents(np.array([57344.0, 57345.0, 1.0]), "e5m2").tolist() == [127, 128, 112]
    for fmt in fp8.FORMATS:
        a = np.exp(np.random.default_rng(1).uniform(-60, 60, 500))
        e = fp8.exponents(a, fmt).astype(float) - 127
        assert (a <= fp8.MAX[fmt] * 2 ** e).all() and (a > fp8.MAX[fmt] * 2 ** (e - 1)).all()


@pytest.mark.parametrize("fmt,half", [("e4m3", 2.0 ** -4), ("e5m2", 2.0 ** -3)])
@pytest.mark.parametrize("block", [1, 128])
def test_restored_values_are_within_half_a_step(fmt, half, block):
    rng = np.random.default_rng(2)
    v = rng.standard_normal((200, 300)) * np.exp(rng.standard_normal((200, 1)))
    codes, e = fp8.pack(v, block, fmt)
    assert e.shape == (3, 200 if block == 1 else 2)
    back = fp8.unpack(codes, e, block, fmt)
    step = np.repeat(np.repeat(2.0 ** (e.astype(float) - 127).T, block, 0)[:200], 128, 1)[:, :300]
    tiny = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}[fmt]
    assert (np.abs(back - v) <= np.maximum(half * np.abs(v), tiny * step)).all()


def test_transposed_groups_are_whole_runs():
    v = np.arange(20.0)[:, None] + np.zeros((20, 3))
    t, used = fp8.transposed(v, np.array([1, 4, 4, 19]))
    assert t.shape == (3, fp8.columns(20, 3)) and used == 256
    assert t[0, :3].tolist() == [1, 2, 3] and not t[0, 3:128].any() and t[0, 128:143].tolist() == list(range(4, 19))


def test_expert_sort_and_gradients_by_definition():
    ids = np.array([[2, 0], [0, -1], [5, 2], [2, 2]])
    off, pos, order = expert.sort(ids, 4)
    assert off.tolist() == [0, 2, 2, 6, 6] and order.tolist() == [1, 2, 0, 5, 6, 7]
    assert pos.tolist() == [[2, 0], [1, -1], [-1, 3], [4, 5]]
    rng = np.random.default_rng(0)
    rows, w, dy = rng.standard_normal((6, 3)), rng.standard_normal((4, 2)), rng.standard_normal((4, 3))
    drows, dw, _ = expert.combine_backward(dy, pos, rows, w)
    loss = lambda r, ww: (dy * expert.combine(r, pos, ww)[0]).sum()  # noqa: E731
    h = 1e-5
    for i in np.ndindex(rows.shape):
        d = np.zeros_like(rows)
        d[i] = h
        assert abs((loss(rows + d, w) - loss(rows - d, w)) / (2 * h) - drows[i]) < 1e-8
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(rows, w + d) - loss(rows, w - d)) / (2 * h) - dw[i]) < 1e-8
    x = rng.standard_normal((4, 3))
    got = expert.gather(x, pos, np.full((6, 3), 9.0))
    assert np.array_equal(got[[0, 1, 2, 3, 4, 5]], x[[0, 1, 0, 2, 3, 3]])
