"""GPU results of sorting slots by expert and of bringing rows there and back
against the fp64 oracle (oracle/expert.py): places bit for bit, sums within
gamma(slots) (dweights: gamma(columns)) of the sums of absolute terms, u =
2^-23, and one rounding to bf16 of half a step, 2^-8."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import expert, fp8
from oracle.muon import bf16_bits_to_f64, f64_to_bf16_bits
from fp8_common import DEV, host
from linear_common import TINY, U, gamma, rounded

pytestmark = pytest.mark.gpu


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _bits(shape, seed):
    return f64_to_bf16_bits(np.random.default_rng(seed).standard_normal(shape))


def _up(bits):
    return bf16_bits_to_f64(bits).reshape(bits.shape)


def _dev(bits, pad=0, shift=0):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16))
    rows, cols = t.shape
    flat = torch.full((shift + rows * (cols + pad) + 64,), 0x7FC0, dtype=torch.int16)
    flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = t
    return torch.as_strided(flat.to(DEV), t.shape, (cols + pad, 1), shift).view(torch.bfloat16)


def _out(rows, cols, pad=0, shift=0):
    import torch
    flat = torch.full((shift + rows * (cols + pad) + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    return torch.as_strided(flat, (rows, cols), (cols + pad, 1), shift), flat


def _untouched(flat, view):
    import torch
    mark = torch.full_like(flat, 7.0)
    torch.as_strided(mark, view.shape, view.stride(), view.storage_offset()).copy_(view)
    return torch.equal(mark.view(torch.int16), flat.view(torch.int16))


def _host(t):
    import torch
    torch.cuda.synchronize()
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def _within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])


def _ids(T, k, E, seed, dropped=0.1):
    rng = np.random.default_rng(seed)
    ids = (rng.random((T, k)) ** 2 * E).astype(np.int64)  # low experts more often, twice for a token too
    out = rng.random((T, k)) < dropped
    ids[out] = rng.choice([-1, E, E + 5, -(2 ** 31)], int(out.sum()))
    return ids


@pytest.mark.parametrize("T,k,E,dropped", [
    (1, 1, 1, 0), (1, 8, 256, 0), (3, 2, 2, 0.5), (64, 1, 7, 0), (65, 3, 5, 0.1), (511, 8, 256, 0.02), (513, 8, 300, 0),
    (2049, 4, 128, 0.05), (5000, 8, 256, 0), (700, 64, 4096, 0.1), (4097, 1, 1500, 0.1), (40000, 2, 33, 0.9), (300, 5, 4, 1.0),
])
@pytest.mark.parametrize("wide", [True, False])
def test_sort(T, k, E, dropped, wide):
    import torch
    ve = _ve()
    print(f"[gpu] expert sort {T}x{k} over {E}", flush=True)
    ids = _ids(T, k, E, T + k + E, dropped)
    off, pos, order = expert.sort(ids, E)
    e = torch.from_numpy(ids if wide else ids.astype(np.int32)).to(DEV)
    o = torch.full((E + 1,), 77, dtype=torch.int64, device=DEV)
    p = torch.full((T, k), 77, dtype=torch.int32, device=DEV)
    r = torch.full((T * k,), 77, dtype=torch.int32, device=DEV)
    for order_out in (r, None):
        ve.expert_sort(e, o, p, order=order_out)
        torch.cuda.synchronize()
        assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(p.cpu().numpy(), pos)
        o.fill_(77)
        p.fill_(77)
    assert np.array_equal(r[:len(order)].cpu().numpy(), order) and bool((r[len(order):] == 77).all())


def test_sort_of_int64_beyond_32_bits_and_of_no_tokens():
    import torch
    ve = _ve()
    ids = np.array([[2 ** 32 + 1, 1], [-(2 ** 32), 0]])   # low words 1 and 0
    o, p = torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    ve.expert_sort(torch.from_numpy(ids).to(DEV), o, p)
    assert o.cpu().tolist() == [0, 1, 2] and p.cpu().tolist() == [[-1, 1], [-1, 0]]
    o.fill_(5)
    ve.expert_sort(torch.empty(0, 4, dtype=torch.int64, device=DEV), o, torch.empty(0, 4, dtype=torch.int32, device=DEV))
    assert o.cpu().tolist() == [0, 0, 0]


def _case(T, k, E, C, seed, spare=3):
    """Positions of a sort, with some rows behind the last place."""
    ids = _ids(T, k, E, seed)
    _, pos, order = expert.sort(ids, E)
    return pos, len(order) + spare


ROWS = [  # tokens, slots, experts, columns, pad, shift
    (1, 1, 1, 1, 0, 0), (1, 8, 16, 4096, 0, 0), (9, 2, 3, 7, 1, 0), (40, 3, 5, 129, 0, 1), (64, 4, 32, 2880, 0, 0),
    (33, 8, 8, 2056, 8, 8), (17, 64, 100, 72, 0, 0), (12, 9, 7, 2049, 3, 5),
]


@pytest.mark.parametrize("T,k,E,C,pad,shift", ROWS)
@pytest.mark.parametrize("weighted", [False, True])
def test_gather(T, k, E, C, pad, shift, weighted):
    import torch
    ve = _ve()
    print(f"[gpu] gather {T}x{k} {C} weighted {weighted}", flush=True)
    pos, R = _case(T, k, E, C, T + C)
    xb = _bits((T, C), 1)
    w = np.random.default_rng(2).standard_normal((T, k)).astype(np.float32) if weighted else None
    out, flat = _out(R, C, pad, shift)
    ve.expert_gather(_dev(xb, pad, shift), torch.from_numpy(pos).to(DEV), out,
                     weights=None if w is None else torch.from_numpy(w).to(DEV))
    ref = expert.gather(_up(xb), pos, np.full((R, C), 7.0), w)
    got = _host(out)
    if weighted:
        _within(got, ref, rounded(U * np.abs(ref), ref), "rows")
    else:
        assert np.array_equal(got, ref)
    assert _untouched(flat, out)


@pytest.mark.parametrize("T,k,E,C,pad,shift", ROWS)
@pytest.mark.parametrize("fmt", fp8.FORMATS)
def test_gather_in_8_bits_equals_packing_the_rows(T, k, E, C, pad, shift, fmt):
    import torch
    ve = _ve()
    pos, R = _case(T, k, E, C, T + C)
    xb = _bits((T, C), 1)
    xb[0, 0] = 0x7F80                                     # an infinity
    out = ve.new_fp8(R, C, 1, fmt, device=DEV)
    for t in (out.codes.view(torch.uint8), out.scales):
        torch.as_strided(t, (t.untyped_storage().nbytes(),), (1,), 0).fill_(0x5A)
    ve.expert_gather(_dev(xb, pad, shift), torch.from_numpy(pos).to(DEV), out)
    codes, e = fp8.pack(_up(xb), 1, fmt)
    got, ge = host(out)
    want, we = np.full((R, C), 0x5A, np.uint8), np.full((e.shape[0], R), 0x5A, np.uint8)
    for t, _, p in expert.slots(pos, R):
        want[p], we[:, p] = codes[t], e[:, t]
    assert np.array_equal(got, want) and np.array_equal(ge, we)
    c = out.codes.view(torch.uint8)
    whole = torch.as_strided(c, (R, -(-C // 16) * 16), (c.stride(0), 1), 0)[:, C:].cpu().numpy()
    filled = np.isin(np.arange(R), pos)
    assert not whole[filled].any() and (whole[~filled] == 0x5A).all()


@pytest.mark.parametrize("T,k,E,C,pad,shift", ROWS)
@pytest.mark.parametrize("weighted,residual", [(True, None), (True, "apart"), (False, None), (False, "in place")])
def test_combine(T, k, E, C, pad, shift, weighted, residual):
    import torch
    ve = _ve()
    print(f"[gpu] combine {T}x{k} {C}", flush=True)
    pos, R = _case(T, k, E, C, T + C)
    rb, sb = _bits((R, C), 1), _bits((T, C), 2) if residual else None
    w = np.random.default_rng(2).standard_normal((T, k)).astype(np.float32) if weighted else None
    if weighted:
        w[pos < 0] = np.nan                               # a slot left out adds nothing, whatever its weight
    y, flat = _out(T, C, pad, shift)
    r = None if sb is None else _dev(sb, pad, shift)
    if residual == "in place":
        y.copy_(r)
        r = y
    ve.expert_combine(_dev(rb, pad, shift), torch.from_numpy(pos).to(DEV), y,
                      weights=None if w is None else torch.from_numpy(w).to(DEV), residual=r)
    ref, mag = expert.combine(_up(rb), pos, w, None if sb is None else _up(sb))
    _within(_host(y), ref, rounded(gamma(k + 1) * mag, ref), "y")
    assert _untouched(flat, y)


@pytest.mark.parametrize("T,k,E,C,pad,shift", ROWS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward(T, k, E, C, pad, shift, weighted):
    import torch
    ve = _ve()
    print(f"[gpu] combine backward {T}x{k} {C}", flush=True)
    pos, R = _case(T, k, E, C, T + C)
    rb, db = _bits((R, C), 1), _bits((T, C), 2)
    w = np.random.default_rng(2).standard_normal((T, k)).astype(np.float32) if weighted else None
    ref, rdw, mag = expert.combine_backward(_up(db), pos, _up(rb), w)
    none = np.isnan(ref)
    ref[none] = 7.0
    p, dw8 = torch.from_numpy(pos).to(DEV), None if w is None else torch.from_numpy(w).to(DEV)
    for parts in ("both", "rows", "weights"):
        out, flat = _out(R, C, pad, shift)
        dw = torch.full((T, k), 7.0, device=DEV)
        ve.expert_combine_backward(_dev(db, pad, shift), p, rows=_dev(rb, pad, shift) if parts != "rows" else None, weights=dw8,
                                   drows=out if parts != "weights" else None, dweights=dw if parts != "rows" else None)
        got = _host(out)
        if parts == "weights":
            assert (got == 7).all()
        else:
            _within(got, ref, np.where(none, 0, rounded(U * np.abs(ref), ref)), "drows")
        assert _untouched(flat, out)
        if parts == "rows":
            assert bool((dw == 7).all())
        else:
            _within(_host(dw), rdw, gamma(C + 8) * mag + TINY, "dweights")


def test_gradients_are_difference_quotients():
    """Small whole numbers: every value is exact in bf16, and so are the
    differences of the sum of y dy."""
    import torch
    ve = _ve()
    rng = np.random.default_rng(0)
    T, k, C = 5, 3, 24
    pos, R = _case(T, k, 4, C, 1)
    rows, dy = rng.integers(-3, 4, (R, C)).astype(float), rng.integers(-2, 3, (T, C)).astype(float)
    w = rng.integers(-2, 3, (T, k)).astype(np.float32)
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).to(DEV)  # noqa: E731
    p = torch.from_numpy(pos).to(DEV)

    def loss(rows, w):
        y = torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
        ve.expert_combine(dev(rows), p, y, weights=torch.from_numpy(w).to(DEV))
        return (y.double().cpu().numpy() * dy).sum()

    drows, dw = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV), torch.empty(T, k, device=DEV)
    ve.expert_combine_backward(dev(dy), p, rows=dev(rows), weights=torch.from_numpy(w).to(DEV), drows=drows, dweights=dw)
    for i in list(np.ndindex(R, C))[::5]:
        d = np.zeros_like(rows)
        d[i] = 1
        assert (loss(rows + d, w) - loss(rows - d, w)) / 2 == _host(drows)[i]
    for i in np.ndindex(T, k):
        d = np.zeros_like(w)
        d[i] = 1
        assert (loss(rows, w + d) - loss(rows, w - d)) / 2 == _host(dw)[i]


def test_positions_outside_the_rows_are_left_out():
    import torch
    ve = _ve()
    C = 40
    pos = torch.tensor([[0, 5], [2 ** 31 - 1, -(2 ** 31)], [2, -1]], dtype=torch.int32, device=DEV)
    x = torch.ones(3, C, dtype=torch.bfloat16, device=DEV)
    rows = torch.full((3, C), 7.0, dtype=torch.bfloat16, device=DEV)
    ve.expert_gather(x, pos, rows)
    assert rows[:, 0].float().cpu().tolist() == [1, 7, 1]
    q = ve.new_fp8(3, C, device=DEV)
    ve.expert_gather(x, pos, q)
    assert q.scales[0].cpu().tolist() == [119, 0, 119]
    y = torch.empty(3, C, dtype=torch.bfloat16, device=DEV)
    ve.expert_combine(rows, pos, y)
    assert y[:, 0].float().cpu().tolist() == [1, 0, 1]
    dw = torch.full((3, 2), 9.0, device=DEV)
    ve.expert_combine_backward(x, pos, rows=rows, drows=rows.clone(), dweights=dw)
    assert dw.cpu().tolist() == [[C, 0], [0, 0], [C, 0]]


def test_infinities_and_nan_pass_through():
    import torch
    ve = _ve()
    pos = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device=DEV)
    rows = torch.ones(4, 16, dtype=torch.bfloat16, device=DEV)
    rows[0, 0], rows[1, 1], rows[2, 2], rows[3] = float("inf"), float("nan"), float("-inf"), float("nan")
    y = torch.empty(2, 16, dtype=torch.bfloat16, device=DEV)
    ve.expert_combine(rows, pos, y, weights=torch.tensor([[2.0, 1.0], [1.0, float("nan")]], device=DEV))
    y = y.float().cpu()
    assert y[0, 0] == float("inf") and torch.isnan(y[0, 1]) and y[0, 3] == 3 and y[1, 2] == float("-inf") and y[1, 0] == 1


def _calls(seed=0, T=700, k=4, E=20, C=264):
    import torch
    ve = _ve()
    ids = torch.from_numpy(_ids(T, k, E, seed)).to(DEV)
    x = _dev(_bits((T, C), seed))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    w = torch.rand(T, k, generator=g, device=DEV)
    off, pos = torch.zeros(E + 1, dtype=torch.int64, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    order = torch.zeros(T * k, dtype=torch.int32, device=DEV)
    rows, y = torch.zeros(T * k, C, dtype=torch.bfloat16, device=DEV), torch.zeros(T, C, dtype=torch.bfloat16, device=DEV)
    drows, dw, q = torch.zeros_like(rows), torch.zeros(T, k, device=DEV), ve.new_fp8(T * k, C, device=DEV)

    def call(**kw):
        ve.expert_sort(ids, off, pos, order=order, **kw)
        ve.expert_gather(x, pos, rows, **kw)
        ve.expert_gather(x, pos, q, **kw)
        ve.expert_combine(rows, pos, y, weights=w, residual=x, **kw)
        ve.expert_combine_backward(y, pos, rows=rows, weights=w, drows=drows, dweights=dw, **kw)

    return call, [off, pos, order, rows, y, drows, dw, q.codes.view(torch.uint8), q.scales]


def test_streams_and_captured_graphs():
    import torch
    call, outs = _calls()
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream(DEV)
    for stream in (None, s, s.cuda_stream):
        for t in outs:
            t.fill_(0)
        s.wait_stream(torch.cuda.current_stream())
        call(stream=stream)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in outs:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    import torch
    pairs = [_calls(seed=2) for _ in range(2)]
    pairs[0][0]()
    torch.cuda.synchronize()
    want = [t.clone() for t in pairs[0][1]]
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for _ in range(5):
        for (call, _), s in zip(pairs, streams):
            call(stream=s)
    torch.cuda.synchronize()
    for _, outs in pairs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_sort_takes_its_workspace():
    import torch
    ve = _ve()
    T, k, E = 3000, 4, 64
    ids = torch.from_numpy(_ids(T, k, E, 1)).to(DEV)
    off, pos = torch.zeros(E + 1, dtype=torch.int64, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    need = ve.expert_sort_workspace(T, k, E)
    assert need > 0
    with pytest.raises(ve.VeError, match="workspace"):
        ve.expert_sort(ids, off, pos, workspace=torch.empty(need - 4, dtype=torch.uint8, device=DEV))
    ve.expert_sort(ids, off, pos, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV))
    ref = expert.sort(ids.cpu().numpy(), E)
    assert np.array_equal(off.cpu().numpy(), ref[0]) and np.array_equal(pos.cpu().numpy(), ref[1])


def test_many_slots():
    """A million slots: chunks of more than one batch a lane."""
    import torch
    ve = _ve()
    T, k, E = 150000, 8, 256
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    off, pos = torch.zeros(E + 1, dtype=torch.int64, device=DEV), torch.zeros(T, k, dtype=torch.int32, device=DEV)
    order = torch.full((T * k,), 77, dtype=torch.int32, device=DEV)
    ve.expert_sort(ids, off, pos, order=order)
    flat = ids.cpu().numpy().reshape(-1)
    n = int((flat >= 0).sum())
    key = np.where(flat >= 0, flat, E)
    want = np.argsort(key, kind="stable")[:n]
    assert np.array_equal(order[:n].cpu().numpy(), want) and bool((order[n:] == 77).all())
    place = np.full(T * k, -1)
    place[want] = np.arange(n)
    assert np.array_equal(pos.cpu().numpy().reshape(-1), place)
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]))


def test_rows_beyond_32_bits():
    """Rows past 4 GiB (and 2^31 elements): the last ones."""
    import torch
    ve = _ve()
    T, k, C = 40000, 8, 7168
    R = T * k                                              # 4.6 GB of rows
    pos = torch.arange(R, dtype=torch.int32, device=DEV).flip(0).view(T, k).contiguous()
    x = torch.arange(T, device=DEV).remainder(128).to(torch.bfloat16)[:, None].expand(T, C).contiguous()
    rows = torch.zeros(R, C, dtype=torch.bfloat16, device=DEV)
    ve.expert_gather(x, pos, rows)
    want = torch.arange(T, device=DEV).remainder(128).flip(0).repeat_interleave(k).to(torch.bfloat16)
    assert torch.equal(rows[:, 0], want) and torch.equal(rows[:, -1], want)
    y = torch.empty_like(x)
    ve.expert_combine(rows, pos, y)
    assert torch.equal(y, (x.float() * k).to(torch.bfloat16))
    dw = torch.empty(T, k, device=DEV)
    ve.expert_combine_backward(torch.ones_like(x), pos, rows=rows, dweights=dw)
    assert torch.equal(dw, x[:, :1].float() * C * torch.ones(1, k, device=DEV))
    rows.zero_()
    ve.expert_combine_backward(x, pos, drows=rows)
    assert torch.equal(rows[:, 5], want)
    del rows
    q = ve.new_fp8(R, C, device=DEV)
    ve.expert_gather(x, pos, q)
    back = torch.empty(1000, C, dtype=torch.bfloat16, device=DEV)
    ve.fp8_unpack(ve.Fp8(q.codes[-1000:], q.scales[:, -1000:]), back)
    assert bool((back - want[-1000:, None]).abs().max() <= 8)  # half a step of a value below 128: 2^-4 of it
