"""Layer norm over very many rows and very wide rows, where a sum has
thousands of terms of one sign.

Tolerances: a sum of n fp32 terms of one sign taken one after another is off
by at most n * 2^-24 of itself.  The backward pass adds up to 512 rows a
thread, then a launch's sum to those before it, eight rows of a block, ten
partial rows and a tree of 32, so (512 + launches + 8 + 10 + 5) * 2^-24; each
term's own product adds 2 * 2^-24.  A row too wide for registers is added up
128 entries a thread, up to 128 such sums, a tree of 32 and 32 warps' sums:
(128 + 128 + 5 + 32) * 2^-24.
"""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z

pytestmark = pytest.mark.gpu

DT = {torch.bfloat16: z.DTYPE_BF16, torch.float32: z.DTYPE_F32}
U = 2.0 ** -24
CHUNK = 1 << 24     # entries a step of the 64-bit reference takes


def backward(dy, x, gamma, mean, rstd, dx):
    rows, cols = x.shape
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    work = torch.full((z.zero1_layernorm_workspace(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    z.zero1_layernorm_backward(rows, cols, DT[x.dtype], dy, dy.stride(0), x, x.stride(0), gamma, mean, rstd, dx,
                               dx.stride(0), dg, db, z.DTYPE_F32, work)
    return dg, db


@pytest.mark.parametrize("rows,cols", [(1 << 25, 8), (1 << 25, 3)])
def test_sums_of_one_sign(rows, cols):
    x = torch.full((rows, cols), 0.37, device="cuda")
    dy = torch.full((rows, cols), 0.0101, device="cuda")
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dg, db = backward(dy, x, torch.ones(cols, device="cuda"), mean, rstd, dy)
    d, h = torch.tensor(0.0101).double().item(), torch.tensor(0.37).double().item()
    launches = rows // (512 * 2 * 100) + 1            # at least 100 SMs
    tol = (512 + launches + 8 + 10 + 5 + 2) * U
    assert (db.double() / (d * rows) - 1).abs().max().item() <= tol
    assert (dg.double() / (d * h * rows) - 1).abs().max().item() <= tol
    del x, dy
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,cols,dtype,pad", [
    (1_300_001, 40, torch.bfloat16, 0), (1_300_001, 33, torch.float32, 0),       # a warp a row
    (330_007, 301, torch.float32, 2), (160_001, 1100, torch.bfloat16, 1),         # unaligned: half a block, a block
    (160_003, 1028, torch.float32, 4), (160_001, 2056, torch.bfloat16, 0),        # a block a row
    (90_001, 8201, torch.bfloat16, 0), (157_001, 8193, torch.bfloat16, 0)])      # wider than registers (unaligned)
def test_rows_in_several_launches(rows, cols, dtype, pad):
    """Every row is taken once, whichever launch it falls into."""
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    x = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]
    dy = torch.empty(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]
    step = CHUNK // cols
    for at in range(0, rows, step):
        n = min(step, rows - at)
        x[at:at + n] = randn(n, cols).to(dtype)
        dy[at:at + n] = randn(n, cols).to(dtype)
    gamma = (1 + 0.2 * randn(cols)).to(dtype)
    mean, rstd = 0.1 * randn(rows), 1 + 0.1 * torch.rand(rows, generator=gen, device="cuda")
    dx = torch.full((rows, cols), float("nan"), dtype=dtype, device="cuda")
    dg, db = backward(dy, x, gamma, mean, rstd, dx)
    again = backward(dy, x, gamma, mean, rstd, torch.empty_like(dx))
    assert torch.equal(dg, again[0]) and torch.equal(db, again[1])
    rdg, rdb = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    sg, sb = torch.zeros_like(rdg), torch.zeros_like(rdb)
    tol = 1e-5 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    for at in range(0, rows, step):
        s = slice(at, at + step)
        d, r = dy[s].double(), rstd[s].double()[:, None]
        h = (x[s].double() - mean[s].double()[:, None]) * r
        g = d * gamma.double()
        want = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        assert (dx[s].double() - want).norm().item() <= tol * want.norm().item() + 1e-6 * (r * g).norm().item()
        rdg += (d * h).sum(0)
        rdb += d.sum(0)
        sg += (d * h).square().sum(0)
        sb += d.square().sum(0)
    assert ((dg.double() - rdg).abs() <= 1e-5 * sg.sum().sqrt()).all()
    assert ((db.double() - rdb).abs() <= 1e-5 * sb.sum().sqrt()).all()
    assert (dg.double() - rdg).norm() <= 1e-5 * sg.sum().sqrt() and (db.double() - rdb).norm() <= 1e-5 * sb.sum().sqrt()
    del x, dy, dx
    torch.cuda.empty_cache()


WIDE = (128 + 128 + 5 + 32) * U


def test_widest_row_forward():
    """2^24 entries with a mean a hundred times their spread: the mean's and
    the variance's terms are all of one sign.  rstd takes half the relative
    error of the variance, and a few roundings."""
    cols = 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(1)
    for dtype in (torch.bfloat16, torch.float32):
        x = (1.0101 + 0.01 * torch.randn(2, cols, generator=gen, device="cuda")).to(dtype)
        y, mean, rstd = torch.empty_like(x), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
        z.zero1_layernorm_forward(2, cols, DT[dtype], x, cols, torch.ones(cols, device="cuda").to(dtype), None, 1e-5, y,
                                  cols, mean, rstd)
        d = x.double()
        m = d.mean(1)
        r = 1 / ((d - m[:, None]).square().mean(1) + 1e-5).sqrt()
        assert ((mean.double() - m).abs() <= (WIDE + 2 * U) * m.abs()).all()
        # the mean's own error shifts the variance by its square only
        assert ((rstd.double() - r).abs() <= (WIDE / 2 + 8 * U) * r).all()


def test_widest_row_backward():
    """A gradient of one value: g - mean(g) is the mean's own error, against g."""
    cols = 1 << 24
    x = torch.randn(1, cols, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    dy = torch.full_like(x, 0.0101)
    mean = x.double().mean(1).float()
    rstd = (1 / x.double().var(1, unbiased=False).sqrt()).float()
    dx = torch.empty_like(x)
    dg, db = backward(dy, x, torch.ones(cols, device="cuda"), mean, rstd, dx)
    h = (x.double() - mean.double()) * rstd.double()
    g = dy.double()
    want = rstd.double() * (g - g.mean() - h * (g * h).mean())
    size = (g * rstd.double()).abs().max()
    # mean(g h): its terms' magnitudes add up to below |g|, and h reaches 6
    assert ((dx.double() - want).abs() <= (WIDE + 4 * U) * size * (1 + h.abs())).all()
    assert torch.equal(db, dy[0])
    assert (dg.double() - (g * h)[0]).norm() <= 4 * U * (g * h).norm() + 2 * U * (g * rstd.double() * x.double().abs()).norm()


@pytest.mark.parametrize("cols", [131072, 131073, 200_003, 400_001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_one_and_several_runs(cols, dtype):
    """Around the width past which a row's sums are taken in runs.  Tolerances
    as for narrower rows: 1e-5 of the norm, and a bf16 entry's rounding."""
    rows, tol = 3, 1e-5 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    gamma = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    z.zero1_layernorm_forward(rows, cols, DT[dtype], x, cols, gamma, None, 1e-5, y, cols, mean, rstd)
    d = x.double()
    m = d.mean(1, keepdim=True)
    r = 1 / ((d - m).square().mean(1, keepdim=True) + 1e-5).sqrt()
    want = (d - m) * r * gamma.double()
    assert (y.double() - want).norm() <= tol * want.norm()
    dx = torch.empty_like(x)
    dg, db = backward(dy, x, gamma, mean, rstd, dx)
    h = (d - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy.double() * gamma.double()
    want = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    assert (dx.double() - want).norm() <= tol * want.norm()
    assert (dg.double() - (dy.double() * h).sum(0)).norm() <= 1e-5 * (dy.double() * h).norm()
    assert (db.double() - dy.double().sum(0)).norm() <= 1e-5 * dy.double().norm()
