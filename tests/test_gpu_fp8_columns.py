"""Weight gradients of matrices in 8-bit floating point over millions of
columns: many groups, and rows as far apart as the products take them.  Whole
numbers of few bits, so that every sum is exact."""

from __future__ import annotations

import pytest

from fp8_common import DEV

pytestmark = pytest.mark.gpu


def _ve():
    import ragged_shard_optimizer_amd as ve
    return ve


def _whole(shape, seed):
    import torch
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("tokens,groups", [(40000, 40000), (100000, 65536)])
def test_many_groups(tokens, groups):
    """5.1 and 8.4 million columns."""
    import torch
    ve = _ve()
    N, K = 40, 24
    dy, x = _whole((tokens, N), 1), _whole((tokens, K), 2)
    # some groups empty, some rows before the first group and behind the last
    cut = torch.randint(1, tokens, (groups + 1,), generator=torch.Generator().manual_seed(3)).sort().values
    off = cut.to(DEV)
    columns = ve.fp8_columns(tokens, groups)
    dyt, xt = ve.new_fp8(N, columns, device=DEV), ve.new_fp8(K, columns, device=DEV)
    ve.fp8_pack(dy, None, dyt, offsets=off)
    ve.fp8_pack(x, None, xt, offsets=off)
    e = torch.searchsorted(off, torch.arange(tokens, device=DEV), right=True) - 1
    inside = (e >= 0) & (e < groups)
    want = torch.zeros(groups, N, K, device=DEV)
    want.index_add_(0, e[inside], dy[inside].float()[:, :, None] * x[inside].float()[:, None, :])
    for dtype in (torch.float32, torch.bfloat16):
        for path in (0, 3):
            dw = torch.full((groups, N, K), 7.0, dtype=dtype, device=DEV)
            with ve.options(linear_path=path):
                ve.fp8_linear_backward(dy_t=dyt, x_t=xt, dw=dw, offsets=off, tokens=tokens)
            assert torch.equal(dw, want.to(dtype)), (dtype, path)


@pytest.mark.parametrize("rows,columns,paths", [(256, (1 << 23) - 128, (0, 2, 3)), (136, (1 << 24) - 128, (0, 2, 3))])
def test_longest_rows(rows, columns, paths):
    """Rows of codes at both limits; the last 500 tokens are not zeros, so that
    every tile's last row is read nearly 2^31 bytes from its first."""
    import torch
    ve = _ve()
    dyt, xt = ve.new_fp8(rows, columns, device=DEV), ve.new_fp8(rows, columns, format="e4m3", device=DEV)
    dy, x = _whole((512, rows), 4), _whole((512, rows), 5)
    dy[-12:], x[-12:] = 0, 0
    for q, v in ((dyt, dy), (xt, x)):
        ve.fp8_pack(v, None, ve.Fp8(q.codes[:, -512:], q.scales[-4:]))
    want = (dy.double().T @ x.double()).float()
    for dtype in (torch.float32, torch.bfloat16):
        for path in paths:
            dw = torch.full((rows, rows), 7.0, dtype=dtype, device=DEV)
            with ve.options(linear_path=path):
                ve.fp8_linear_backward(dy_t=dyt, x_t=xt, dw=dw, tokens=columns - 12)
            assert torch.equal(dw, want.to(dtype)), (dtype, path)
