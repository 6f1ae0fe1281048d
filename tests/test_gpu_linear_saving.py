"""GPU: activations saved in 8 bits by the forward product's epilogue, in
every form of the product.

With one 1 in each row of w the product is a selection, z[t, n] = x[t, s(n)],
exact in fp32 whatever the order of the sum, and z + bias is one fp32
addition: scales and codes are then known."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import linear
from oracle.muon import f64_to_bf16_bits
from test_gpu_linear import DEV, _bits, _dev, _forward_case, _up, _ve

pytestmark = pytest.mark.gpu

FORMS = [(0, 1), (1, 0), (1, 1), (2, 0), (2, 1), (3, 0), (3, 1)]

# out_features is a multiple of 8 but not of the run, so that a row's last run
# is short and the tile goes on past the row's end
SHORT_RUNS = [
    # T, K, N, groups, act, bias, residual, z, block, pad, shift
    (40, 99, 136, None, "none", False, False, False, 64, 0, 0),
    (400, 99, 136, None, "silu", False, False, False, 64, 0, 0),
    (400, 131, 520, None, "none", True, False, False, 32, 0, 0),
    (300, 64, 264, None, "gelu", True, False, True, 128, 0, 0),
    (333, 99, 136, 7, "silu", True, False, True, 64, 0, 0),
    (333, 129, 1000, 5, "none", True, False, False, 128, 3, 1),
    (200, 65, 8, None, "relu", True, False, False, 32, 0, 0),
]


@pytest.mark.parametrize("path,split", [(0, 1), (1, 0), (1, 1), (2, 0), (3, 0)])
@pytest.mark.parametrize("case", SHORT_RUNS, ids=lambda c: "-".join(map(str, c)))
def test_short_last_run(case, path, split):
    ve = _ve()
    print(f"[gpu] forward {case} path {path} split {split}", flush=True)
    with ve.options(linear_path=path, linear_split=split):
        _forward_case(*case)


# the form that the shape itself leads to
@pytest.mark.parametrize("case", [
    (1000, 129, 1000, None, "silu", True, False, False, 32, 0, 0),
    (4096, 131, 520, None, "none", True, False, False, 32, 0, 0),
    (8000, 1001, 1000, 64, "none", True, False, False, 128, 0, 0),
], ids=lambda c: "-".join(map(str, c)))
def test_short_last_run_by_shape(case):
    print(f"[gpu] forward {case}", flush=True)
    _forward_case(*case)


def _selection(T, K, N, E, seed, cancel):
    """x, w, bias (bf16 bits), offsets and z (fp32): w picks column n mod K for
    output n.  cancel: the last output's column, the first of x, is 96 to 192
    times the others and its bias takes it away again."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((T, K)) * np.exp(3 * rng.standard_normal((T, 1)))
    bias = 0.2 * rng.standard_normal((E or 1, N))
    pick = np.arange(N) % K
    if cancel:
        pick = 1 + np.arange(N) % (K - 1)
        pick[-1] = 0
        v = rng.uniform(0.5, 1, (T, K)) * np.sign(v)
        v[:, 0] = 96
        bias[:, -1] = -96
    xb, bb = f64_to_bf16_bits(v), f64_to_bf16_bits(bias)
    w = np.zeros((E or 1, N, K))
    w[:, np.arange(N), pick] = 1
    off = None if E is None else np.concatenate([[1], 1 + np.cumsum(rng.multinomial(T - 3, np.ones(E) / E))])
    z = np.full((T, N), np.nan, np.float32)
    for e, a, b in linear.parts(off, T):
        z[a:b] = _up(xb)[a:b, pick].astype(np.float32) + _up(bb)[e].astype(np.float32)
    wb = f64_to_bf16_bits(w)
    return (xb, wb, bb, off, z) if E else (xb, wb[0], bb[0], off, z)


def _saved(xb, wb, bb, off, block):
    import torch
    ve = _ve()
    T, N = xb.shape[0], wb.shape[-2]
    q = ve.new_act8(T, N, block, DEV)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    ve.linear_forward(_dev(xb), _dev(wb), y, bias=_dev(bb), z8=q, offsets=None if off is None else torch.from_numpy(off).to(DEV))
    torch.cuda.synchronize()
    return q.codes.cpu().numpy(), q.scales.cpu().numpy()


@pytest.mark.parametrize("path,split", FORMS)
@pytest.mark.parametrize("T,K,N,E,block", [(70, 99, 136, None, 64), (150, 131, 520, None, 32), (70, 99, 136, 3, 128)])
def test_bias_that_cancels_the_last_column(T, K, N, E, block, path, split):
    """The last output is 0; nothing of its product may reach the scale of its run."""
    ve = _ve()
    print(f"[gpu] cancelled {T} {K} {N} {E} {block} path {path} split {split}", flush=True)
    xb, wb, bb, off, z = _selection(T, K, N, E, 1, True)
    with ve.options(linear_path=path, linear_split=split):
        codes, scales = _saved(xb, wb, bb, off, block)
    inside = ~np.isnan(z).any(1)
    want_c, want_s = linear.pack(z[inside], block)
    # scale to a unit in the last place (2^-23 relative at most), a code to the neighbouring one
    assert np.all(np.abs(scales[inside] - want_s) <= 2.0 ** -23 * want_s)
    assert np.abs(codes[inside].astype(int) - want_c).max() <= 1
