"""What the 8-bit products keep where large products cancel: each of 8
consecutive products loses up to 2^-13 of the largest of the 8 (``cut`` in
tests/fp8_common.py), however small the sum is; an fp32 dw loses nothing there."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import linear
from fp8_common import DEV, cut, device, forward_bounds, packed_values
from linear_common import TINY, gamma, rounded

pytestmark = pytest.mark.gpu
FORMS = (0, 2, 3, 4)  # linear_path: chosen, 128 x 128, 256 x 256, few rows


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _products(x, w):
    """Every way to x w^T ([rows, K] and [cols, K], K a multiple of 128, rows of
    x in blocks of their own): (name, result) of forward and dx in each form and
    of dw, where K are the tokens, in bf16 and fp32."""
    import torch
    ve = _ve()
    T, N, K = x[0].shape[0], w[0].shape[0], x[0].shape[1]
    xq, wq = device(*x[:2]), device(*w[:2], 128)
    rows = device(w[0], np.repeat(w[1], 128, 1)[:, :N])  # w's codes with a scale for each row
    for path in FORMS:
        with ve.options(linear_path=path):
            y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
            ve.fp8_linear_forward(xq, wq, y)
            yield f"forward {path}", _host(y)
            ve.fp8_linear_backward(dy=xq, w_t=wq, dx=y.zero_())
            yield f"dx {path}", _host(y)
            for dtype in (torch.bfloat16, torch.float32):
                dw = torch.empty(T, N, dtype=dtype, device=DEV)
                ve.fp8_linear_backward(dy_t=xq, x_t=rows, dw=dw, tokens=K)
                yield f"dw {path}" + (" fp32" if dtype == torch.float32 else ""), _host(dw)


@pytest.mark.parametrize("apart", [False, True])
def test_one_beside_two_that_cancel(apart):
    """448 448 - 448 448 + 1: 0 within 8 consecutive products, whose cut is 2^4
    (2^17 is the power of two in 448^2), and 1 where the 1 is not one of them."""
    x, w = np.zeros((1, 128)), np.zeros((1, 128))
    x[0, :2], w[0, 0], w[0, 1] = 448, 448, -448
    x[0, 8 if apart else 2] = w[0, 8 if apart else 2] = 1
    x, w = packed_values(x, 1, "e4m3"), packed_values(w, 128, "e4m3")
    for name, got in _products(x, w):
        print(f"[gpu] {name}: {got[0, 0]}", flush=True)
        assert got[0, 0] == (1 if apart or "fp32" in name else 0), name


@pytest.mark.parametrize("T,K,N", [(5, 512, 40), (40, 1024, 136), (300, 512, 264)])
@pytest.mark.parametrize("distance", [1, 8, 128])
def test_outlier_columns_that_cancel(T, K, N, distance):
    """A few columns 2^9 times the rest, in pairs `distance` apart whose products
    cancel: the result is the ordinary columns'."""
    rng = np.random.default_rng(T + distance)
    x, w = rng.standard_normal((T, K)), rng.standard_normal((N, K)) * K ** -0.5
    at = np.arange(3, K - distance, 256 if distance == 128 else 32)
    x[:, at] = 512 * np.sign(x[:, at])
    x[:, at + distance] = x[:, at]
    w[:, at + distance] = -w[:, at]
    x, w = packed_values(x, 1, "e4m3"), packed_values(w, 128, "e4m3")
    ref, z, mag = linear.forward(x[2], w[2])
    lost = cut(x[2], w[2])
    bound = forward_bounds(ref, z, mag, lost, K, "none")[1]
    exact = gamma(K + 130) * mag + TINY
    rms = np.sqrt((ref ** 2).mean())
    for name, got in _products(x, w):
        err = np.abs(got - ref)
        print(f"[gpu] {T}x{K}x{N} pairs {distance} apart, {name}: largest error {err.max() / rms:.2e} of the results' rms", flush=True)
        b = exact if "fp32" in name else rounded(exact + lost, ref) if "dw" in name else bound
        assert (err <= b).all(), (name, float((err / b).max()))
