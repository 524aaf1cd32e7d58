"""Layer norm forward and backward on the GPU against the definition in 64
bits, and the backward pass against differences of the forward definition.

Tolerances, from the arithmetic: fp32 sums of n terms by trees and short runs
stay below 64 * 2^-24 of the sum of magnitudes at these sizes, each output
adds a handful of roundings, so 1e-5 of the output's norm in fp32; a bf16
output adds its own rounding, at most 2^-8 of each entry (8 significant
bits).  The column sums
run over the rows: 1e-5 of the root of the summed squares.
"""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

EPS = 1e-5
DT = {torch.bfloat16: z.DTYPE_BF16, torch.float32: z.DTYPE_F32}
TOL = {torch.float32: 1e-5, torch.bfloat16: 1e-5 + 2.0 ** -8}


def rows_of(rows, cols, pad, dtype, shift=0, guard=True):
    """A Guarded flat buffer and its (rows, cols) view, `shift` entries off alignment."""
    g = Guarded(rows * (cols + pad) + shift, dtype)
    v = torch.as_strided(g.t, (rows, cols), (cols + pad, 1), g.t.storage_offset() + shift)
    return g, v


def rel(got, want):
    n = want.norm().item()
    return (got.double() - want).norm().item() / n if n else got.double().abs().max().item()


def ref_fwd(x, gamma, beta, eps=EPS):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd


def ref_bwd(dy, x, gamma, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    g = dy * gamma.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0), (dy * h).square().sum(0).sqrt().norm().item(), dy.norm().item()


# widths on both sides of every variant's bound, odd ones, and one too wide for registers
COLS = [1, 2, 7, 31, 64, 100, 256, 257, 512, 767, 768, 1000, 1021, 1024, 1025, 2048, 2050, 4096, 4100, 5003, 8192, 8200,
        16384, 16392, 20001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,pad,shift,bias", [(1, 0, 0, True), (13, 0, 0, True), (70, 8, 0, False), (9, 3, 1, True)])
def test_forward_and_backward(rows, cols, pad, shift, bias, dtype):
    gen = torch.Generator(device="cuda").manual_seed(cols * 31 + rows)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    gx, x = rows_of(rows, cols, pad, dtype, shift)
    gy, y = rows_of(rows, cols, pad, dtype, shift)
    x.copy_(randn(rows, cols) * 1.5 + 0.7)
    gamma, beta = (1 + 0.2 * randn(cols)).to(dtype), (0.3 * randn(cols)).to(dtype) if bias else None
    mean, rstd = Guarded(rows, torch.float32), Guarded(rows, torch.float32)
    z.zero1_layernorm_forward(rows, cols, DT[dtype], x, cols + pad, gamma, beta, EPS, y, cols + pad, mean.t, rstd.t)
    ry, rm, rr = ref_fwd(x, gamma, beta)
    # an entry cancels to x - mean: the mean's rounding counts against |x| * rstd
    slack = 4 * 2.0 ** -24 * (x.double().abs().max() * rr.max() * gamma.double().abs().max()).item() * (rows * cols) ** 0.5
    assert (y.double() - ry).norm().item() <= TOL[dtype] * ry.norm().item() + slack
    assert rel(mean.t, rm) <= 1e-5 + 2.0 ** -22 * (x.double().norm() / (cols ** 0.5) / max(rm.norm().item(), 1e-30)).item()
    assert rel(rstd.t, rr) <= 1e-5

    gdy, dy = rows_of(rows, cols, pad, dtype, shift)
    gdx, dx = rows_of(rows, cols, pad, dtype, shift)
    dy.copy_(randn(rows, cols) * 1e-2)
    for gt in (torch.float32, torch.bfloat16):
        dgamma, dbeta = Guarded(cols, gt), Guarded(cols, gt)
        work = Guarded(z.zero1_layernorm_workspace(rows, cols) // 4, torch.float32)
        z.zero1_layernorm_backward(rows, cols, DT[dtype], dy, cols + pad, x, cols + pad, gamma, mean.t, rstd.t, dx,
                                   cols + pad, dgamma.t, dbeta.t if bias else None, DT[gt], work.t)
        rdx, rdg, rdb, sg, sb = ref_bwd(dy, x, gamma, mean.t, rstd.t)
        size = (rstd.t.double()[:, None] * dy.double() * gamma.double()).norm().item()   # dx cancels against this
        assert (dx.double() - rdx).norm().item() <= TOL[dtype] * rdx.norm().item() + 1e-6 * size
        round_g = 0.0 if gt == torch.float32 else 2.0 ** -8
        assert (dgamma.t.double() - rdg).norm().item() <= 1e-5 * sg + round_g * rdg.norm().item()
        if bias:
            assert (dbeta.t.double() - rdb).norm().item() <= 1e-5 * sb + round_g * rdb.norm().item()
        assert dgamma.intact() and dbeta.intact() and work.intact()
    for q in (gx, gy, gdy, gdx, mean, rstd):
        assert q.intact()


@pytest.mark.parametrize("rows,cols,dtype", [(5000, 768, torch.bfloat16), (3001, 1021, torch.float32),
                                             (2000, 4096, torch.bfloat16), (700, 9001, torch.float32)])
def test_many_rows(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * 2 - 1).to(dtype)
    dy = (torch.randn(rows, cols, generator=gen, device="cuda") * 1e-2).to(dtype)
    gamma = torch.randn(cols, generator=gen, device="cuda").to(dtype)
    beta = torch.randn(cols, generator=gen, device="cuda").to(dtype)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(2):
        work.fill_(0xFF)          # nothing is taken from the workspace as it was
        z.zero1_layernorm_forward(rows, cols, DT[dtype], x, cols, gamma, beta, EPS, y, cols, mean, rstd)
        z.zero1_layernorm_backward(rows, cols, DT[dtype], dy, cols, x, cols, gamma, mean, rstd, dx, cols, dg, db,
                                   z.DTYPE_F32, work)
        got.append([t.clone() for t in (y, mean, rstd, dx, dg, db)])
    assert all(torch.equal(a, b) for a, b in zip(*got))      # deterministic
    assert rel(y, ref_fwd(x, gamma, beta)[0]) <= TOL[dtype]
    rdx, rdg, rdb, sg, sb = ref_bwd(dy, x, gamma, mean, rstd)
    assert rel(dx, rdx) <= TOL[dtype]
    assert (dg.double() - rdg).norm().item() <= 1e-5 * sg and (db.double() - rdb).norm().item() <= 1e-5 * sb


@pytest.mark.parametrize("rows,cols", [(3, 5), (4, 96), (2, 1500)])
def test_backward_against_differences(rows, cols):
    """d(sum(y * w))/d(x, gamma, beta) by central differences of the fp64
    definition along random directions: truncation is O(step^2), so 1e-4."""
    gen = torch.Generator(device="cuda").manual_seed(77)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda", dtype=torch.float64)

    x, gamma, beta, w = randn(rows, cols).float(), randn(cols).float(), randn(cols).float(), randn(rows, cols).float()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    z.zero1_layernorm_forward(rows, cols, z.DTYPE_F32, x, cols, gamma, beta, EPS, y, cols, mean, rstd)
    z.zero1_layernorm_backward(rows, cols, z.DTYPE_F32, w, cols, x, cols, gamma, mean, rstd, dx, cols, dg, db,
                               z.DTYPE_F32, work)
    h = 1e-4
    for grad, at in ((dx, 0), (dg, 1), (db, 2)):
        args = [x.double(), gamma.double(), beta.double()]
        for _ in range(3):
            v = randn(*args[at].shape)
            lo, hi = list(args), list(args)
            lo[at], hi[at] = args[at] - h * v, args[at] + h * v
            diff = ((ref_fwd(*hi)[0] - ref_fwd(*lo)[0]) * w.double()).sum() / (2 * h)
            got = (grad.double() * v).sum()
            assert abs((got - diff).item()) <= 1e-4 * (grad.double().norm() * v.norm()).item()


@pytest.mark.parametrize("cols", [96, 3000, 17000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place(cols, dtype):
    rows = 50
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    gamma = torch.randn(cols, generator=gen, device="cuda").to(dtype)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    outs = []
    for inplace in (False, True):
        xi, di = x.clone(), dy.clone()
        y = xi if inplace else torch.empty_like(x)
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        z.zero1_layernorm_forward(rows, cols, DT[dtype], xi, cols, gamma, None, EPS, y, cols, mean, rstd)
        dx = di if inplace else torch.empty_like(x)
        z.zero1_layernorm_backward(rows, cols, DT[dtype], di, cols, x, cols, gamma, mean, rstd, dx, cols, dg, db,
                                   z.DTYPE_F32, work)
        outs.append((y, dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_no_rows_writes_zero_gradients():
    dg, db = torch.full((70,), 3.0, device="cuda"), torch.full((70,), 3.0, device="cuda")
    work = torch.full((z.zero1_layernorm_workspace(0, 70),), 0xFF, dtype=torch.uint8, device="cuda")
    gamma = torch.ones(70, device="cuda")
    empty = torch.empty(0, 70, device="cuda")
    none = torch.empty(0, device="cuda")
    z.zero1_layernorm_backward(0, 70, z.DTYPE_F32, empty, 70, empty, 70, gamma, none, none, empty, 70, dg, db,
                               z.DTYPE_F32, work)
    assert (dg == 0).all() and (db == 0).all()


def test_constant_and_not_finite_rows():
    """A row of one value is beta; an infinity or a NaN stays in its row, and
    reaches only the column sums of the backward pass."""
    x = torch.randn(6, 200, device="cuda")
    x[2] = 7.0
    x[4, 3] = float("inf")
    gamma, beta = torch.randn(200, device="cuda"), torch.randn(200, device="cuda")
    y = torch.empty_like(x)
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    z.zero1_layernorm_forward(6, 200, z.DTYPE_F32, x, 200, gamma, beta, EPS, y, 200, mean, rstd)
    assert torch.equal(y[2], beta)
    assert torch.isnan(y[4]).all()
    keep = [0, 1, 2, 3, 5]
    assert rel(y[keep], ref_fwd(x[keep], gamma, beta)[0]) <= 1e-5


def test_gradients_into_a_flat_buffer_at_an_odd_offset():
    """bf16 weight gradients land at their place in a flat gradient buffer."""
    rows, cols = 40, 65
    flat = Guarded(1000, torch.bfloat16)
    flat.t.fill_(9.0)
    x, dy = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    gamma = torch.randn(cols, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    z.zero1_layernorm_forward(rows, cols, z.DTYPE_F32, x, cols, gamma, None, EPS, y, cols, mean, rstd)
    z.zero1_layernorm_backward(rows, cols, z.DTYPE_F32, dy, cols, x, cols, gamma, mean, rstd, dx, cols,
                               flat.t[301:301 + cols], flat.t[301 + cols:301 + 2 * cols], z.DTYPE_BF16, work)
    _, rdg, rdb, _, _ = ref_bwd(dy, x, gamma, mean, rstd)
    assert rel(flat.t[301:301 + cols], rdg) <= 2.0 ** -8 and rel(flat.t[301 + cols:301 + 2 * cols], rdb) <= 2.0 ** -8
    assert (flat.t[:301].float() == 9).all() and (flat.t[301 + 2 * cols:].float() == 9).all() and flat.intact()


@pytest.mark.parametrize("cols", [96, 1001])
def test_rows_past_32_bits(cols):
    """Rows so far apart that the last begins beyond 2^32 entries; forward and
    backward in place."""
    rows, ld = 3, (1 << 31) + 8
    full = torch.zeros((rows - 1) * ld + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(full, (rows, cols), (ld, 1))
    keep = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
    x.copy_(keep)
    gamma = torch.randn(cols, device="cuda").to(torch.bfloat16)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    z.zero1_layernorm_forward(rows, cols, z.DTYPE_BF16, x, ld, gamma, None, EPS, x, ld, mean, rstd)
    ry, rm, rr = ref_fwd(keep, gamma, None)
    assert rel(x, ry) <= TOL[torch.bfloat16] and rel(rstd, rr) <= 1e-5
    dy = torch.randn(rows, cols, device="cuda").to(torch.bfloat16)
    x.copy_(dy)                                   # dy, and dx in its place
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    z.zero1_layernorm_backward(rows, cols, z.DTYPE_BF16, x, ld, keep, cols, gamma, mean, rstd, x, ld, dg, db,
                               z.DTYPE_F32, work)
    rdx, rdg, rdb, sg, sb = ref_bwd(dy, keep, gamma, mean, rstd)
    assert rel(x, rdx) <= TOL[torch.bfloat16]
    assert (dg.double() - rdg).norm().item() <= 1e-5 * sg and (db.double() - rdb).norm().item() <= 1e-5 * sb
    del full, x
    torch.cuda.empty_cache()
