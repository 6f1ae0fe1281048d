"""What the operators write, on buffers that hold something else before: the
weight gradient's empty groups past 32-bit offsets, and rows by expert on two
streams at once."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import expert, fp8
from oracle.muon import f64_to_bf16_bits
from fp8_common import DEV, cut, device, packed_values
from linear_common import TINY, gamma, rounded

pytestmark = pytest.mark.gpu


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def test_empty_groups_beyond_32_bits_become_zeros():
    """4.4 G elements of dw, every one of them written: those of groups without
    rows as zeros."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(0)
    K, N, E, last = 8192, 8192, 66, 40
    off = np.zeros(E + 1, np.int64)
    off[E] = last
    dw = torch.full((E, N, K), 3.0, dtype=torch.bfloat16, device=DEV)
    dyc, dye, dyv = packed_values(fp8.transposed(rng.standard_normal((last, N)), off)[0], 1, "e4m3")
    xtc, xte, xv = packed_values(fp8.transposed(rng.standard_normal((last, K)), off)[0], 1, "e4m3")
    ve.fp8_linear_backward(dy_t=device(dyc, dye), x_t=device(xtc, xte), dw=dw, offsets=torch.from_numpy(off).to(DEV), tokens=last)
    assert all(bool((dw[e] == 0).all()) for e in range(E - 1))
    for at in (0, N - 64):
        a = dyv[at:at + 64, :128]
        ref, mag = a @ xv[:, :128].T, np.abs(a) @ np.abs(xv[:, :128]).T
        got = dw[-1, at:at + 64].double().cpu().numpy()
        bound = rounded(gamma(last + 130) * mag + cut(a, xv[:, :128]) + TINY, ref)
        assert (np.abs(got - ref) <= bound).all()


@pytest.mark.parametrize("T,k,E,C", [(700, 4, 20, 264), (3000, 8, 130, 72)])
def test_rows_by_expert_on_two_streams_at_once(T, k, E, C):
    """Each stream's outputs start from markers; the results are the oracle's."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E + 1, (T, k))
    off, pos, order = expert.sort(ids, E)[:3]
    n = int(off[-1])
    bits = f64_to_bf16_bits(rng.standard_normal((T, C)))
    x = torch.from_numpy(bits.view(np.int16)).to(DEV).view(torch.bfloat16)
    dev_ids = torch.from_numpy(ids).to(DEV)
    sides = []
    for _ in range(2):
        sides.append(dict(
            off=torch.full((E + 1,), -7, dtype=torch.int64, device=DEV), pos=torch.full((T, k), -7, dtype=torch.int32, device=DEV),
            order=torch.full((T * k,), -7, dtype=torch.int32, device=DEV),
            rows=torch.full((T * k, C), 7.0, dtype=torch.bfloat16, device=DEV),
            q=ve.new_fp8(T * k, C, device=DEV), back=torch.full((T * k, C), 7.0, dtype=torch.bfloat16, device=DEV),
            stream=torch.cuda.Stream(DEV)))
    torch.cuda.synchronize()
    for _ in range(3):
        for s in sides:
            kw = dict(stream=s["stream"])
            ve.expert_sort(dev_ids, s["off"], s["pos"], order=s["order"], **kw)
            ve.expert_gather(x, s["pos"], s["rows"], **kw)
            ve.expert_gather(x, s["pos"], s["q"], **kw)
            ve.fp8_unpack(s["q"], s["back"], **kw)
    torch.cuda.synchronize()
    want = torch.from_numpy(bits.view(np.int16)[np.asarray(order[:n]) // k]).to(DEV).view(torch.bfloat16)
    codes, e = fp8.pack(x.double().cpu().numpy()[np.asarray(order[:n]) // k])
    eight = torch.from_numpy(fp8.unpack(codes, e)).to(torch.bfloat16).to(DEV)
    for s in sides:
        assert np.array_equal(s["off"].cpu().numpy(), off) and np.array_equal(s["pos"].cpu().numpy(), pos)
        assert np.array_equal(s["order"].cpu().numpy()[:n], order[:n]) and bool((s["order"][n:] == -7).all())
        assert torch.equal(s["rows"][:n], want) and bool((s["rows"][n:] == 7).all())
        assert torch.equal(s["back"][:n], eight) and not bool(s["back"][n:].any())
