"""Layer norm whose operands differ in stride and alignment from one another,
and weight gradients in bf16 over a whole batch.

Tolerances as in test_gpu_layernorm.py: 1e-5 of the norm, and 2^-8 of it where
an entry is rounded to bf16.
"""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

DT = {torch.bfloat16: z.DTYPE_BF16, torch.float32: z.DTYPE_F32}
TOL = {torch.float32: 1e-5, torch.bfloat16: 1e-5 + 2.0 ** -8}
NAMES = ["x", "y", "dy", "dx", "gamma", "beta"]


def operand(rows, cols, dtype, odd):
    """A guarded (rows, cols) view: dense and aligned, or one entry off with rows a few entries apart."""
    pad, shift = (3, 1) if odd else (0, 0)
    g = Guarded(rows * (cols + pad) + shift, dtype)
    return g, torch.as_strided(g.t, (rows, cols), (cols + pad, 1), g.t.storage_offset() + shift), cols + pad


@pytest.mark.parametrize("odd", [()] + [(n,) for n in NAMES] + [("y", "dx"), ("x", "dy"), ("dy", "gamma")])
@pytest.mark.parametrize("cols", [256, 768, 1024, 4096, 8208, 16384, 18432])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_each_operand_by_itself(odd, cols, dtype):
    rows = 37
    gen = torch.Generator(device="cuda").manual_seed(cols)

    def randn(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    held = {n: operand(rows if n not in ("gamma", "beta") else 1, cols, dtype, n in odd) for n in NAMES}
    t, ld = {n: h[1] for n, h in held.items()}, {n: h[2] for n, h in held.items()}
    t["x"].copy_(randn(rows, cols) * 1.5 + 0.2)
    t["dy"].copy_(randn(rows, cols) * 1e-2)
    t["gamma"].copy_(1 + 0.2 * randn(1, cols))
    t["beta"].copy_(0.3 * randn(1, cols))
    gamma, beta = t["gamma"][0], t["beta"][0]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    z.zero1_layernorm_forward(rows, cols, DT[dtype], t["x"], ld["x"], gamma, beta, 1e-5, t["y"], ld["y"], mean, rstd)
    x = t["x"].double()
    m = x.mean(1, keepdim=True)
    r = 1 / ((x - m).square().mean(1, keepdim=True) + 1e-5).sqrt()
    want = (x - m) * r * gamma.double() + beta.double()
    assert (t["y"].double() - want).norm() <= TOL[dtype] * want.norm()
    dg, db = Guarded(cols, torch.float32), Guarded(cols, torch.float32)
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    z.zero1_layernorm_backward(rows, cols, DT[dtype], t["dy"], ld["dy"], t["x"], ld["x"], gamma, mean, rstd, t["dx"],
                               ld["dx"], dg.t, db.t, z.DTYPE_F32, work)
    h = (x - mean.double()[:, None]) * rstd.double()[:, None]
    d = t["dy"].double()
    g = d * gamma.double()
    want = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    assert (t["dx"].double() - want).norm() <= TOL[dtype] * want.norm()
    assert (dg.t.double() - (d * h).sum(0)).norm() <= 1e-5 * (d * h).norm()
    assert (db.t.double() - d.sum(0)).norm() <= 1e-5 * d.norm()
    assert all(q[0].intact() for q in held.values()) and dg.intact() and db.intact()


@pytest.mark.parametrize("rows,cols", [(16384, 768), (4096, 4096), (3001, 1021)])
def test_bf16_weight_gradients_of_a_batch_in_the_flat_buffer(rows, cols):
    """The gradients an optimizer step reads: bf16, at their place among other parameters'."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(torch.bfloat16)
    dy = (1e-2 * torch.randn(rows, cols, generator=gen, device="cuda")).to(torch.bfloat16)
    gamma = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    z.zero1_layernorm_forward(rows, cols, z.DTYPE_BF16, x, cols, gamma, None, 1e-5, y, cols, mean, rstd)
    flat = Guarded(4 * cols, torch.bfloat16)
    flat.t.fill_(9.0)
    work = torch.empty(z.zero1_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    exact = [torch.empty(cols, device="cuda") for _ in range(2)]
    for dg, db, kind in ((flat.t[cols:2 * cols], flat.t[2 * cols:3 * cols], z.DTYPE_BF16), (*exact, z.DTYPE_F32)):
        z.zero1_layernorm_backward(rows, cols, z.DTYPE_BF16, dy, cols, x, cols, gamma, mean, rstd, dx, cols, dg, db, kind,
                                   work)
    # one rounding of the fp32 sums
    assert torch.equal(flat.t[cols:2 * cols], exact[0].to(torch.bfloat16))
    assert torch.equal(flat.t[2 * cols:3 * cols], exact[1].to(torch.bfloat16))
    assert (flat.t[:cols].float() == 9).all() and (flat.t[3 * cols:].float() == 9).all() and flat.intact()
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    assert (exact[0].double() - (dy.double() * h).sum(0)).norm() <= 1e-5 * (dy.double() * h).norm()
    assert (exact[1].double() - dy.double().sum(0)).norm() <= 1e-5 * dy.double().norm()
