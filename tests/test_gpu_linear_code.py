"""GPU: the 8-bit code of the forward product's epilogue is the rule's, bit for
bit, in every form of the product (products that are selections, so that the
saved values are known exactly)."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import linear
from oracle.muon import bf16_bits_to_f64, f64_to_bf16_bits
from test_gpu_linear import DEV, _dev, _up, _ve
from test_gpu_linear_saving import FORMS, _saved, _selection

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path,split", FORMS)
@pytest.mark.parametrize("T,K,N,E,block", [
    (300, 64, 136, None, 64), (300, 99, 136, None, 64), (257, 640, 520, None, 32), (300, 72, 264, 5, 128),
    (300, 99, 75, 5, 32),
])
def test_code_of_the_epilogue(T, K, N, E, block, path, split):
    ve = _ve()
    print(f"[gpu] code {T} {K} {N} {E} {block} path {path} split {split}", flush=True)
    xb, wb, bb, off, z = _selection(T, K, N, E, 2, False)
    with ve.options(linear_path=path, linear_split=split):
        codes, scales = _saved(xb, wb, bb, off, block)
    inside = ~np.isnan(z).any(1)
    want_c, want_s = linear.pack(z[inside], block)
    assert np.array_equal(scales[inside].view(np.uint32), want_s.view(np.uint32))
    assert np.array_equal(codes[inside], want_c)


@pytest.mark.parametrize("path", [1, 2, 3])
def test_code_of_every_bf16_magnitude(path):
    """Runs for each positive normal bf16 value as its largest magnitude, in
    waves of one kind and in mixed ones."""
    import torch
    ve = _ve()
    print(f"[gpu] code of every magnitude, path {path}", flush=True)
    amax = np.arange(0x80, 0x7F80, dtype=np.uint16)
    w = np.eye(128)
    for order in (np.arange(len(amax)), np.random.default_rng(0).permutation(len(amax))):
        a = bf16_bits_to_f64(amax[order])
        v = a[:, None] * np.random.default_rng(1).uniform(0.01, 1, (len(a), 128))
        v[np.abs(v) < 2.0 ** -126] = 0                 # the matrix units may take subnormal inputs as 0
        v[:, 7], v[:, 39], v[:, 64], v[:, 127] = a, -a, a, -a
        bits = f64_to_bf16_bits(v)
        codes, scales = linear.pack(_up(bits).astype(np.float32), 32)
        q = ve.new_act8(len(a), 128, 32, DEV)
        with ve.options(linear_path=path):
            ve.linear_forward(_dev(bits), _dev(f64_to_bf16_bits(w)), torch.empty(len(a), 128, dtype=torch.bfloat16, device=DEV),
                              z8=q)
        torch.cuda.synchronize()
        assert np.array_equal(q.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
        assert np.array_equal(q.codes.cpu().numpy(), codes)
