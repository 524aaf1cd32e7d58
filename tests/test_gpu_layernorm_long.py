"""Layer norm over very many rows and very wide rows, where a sum has
thousands of terms of one sign.

Tolerances: a sum of n fp32 terms of one sign taken one after another is off
by at most n * 2^-24 of itself.  The backward pass adds up to 512 rows a
thread, then a launch's sum to those before it, eight rows of a block, ten
partial rows and a tree of 32, so (512 + launches + 8 + 10 + 5) * 2^-24; each
term's own product adds 2 * 2^-24.
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
