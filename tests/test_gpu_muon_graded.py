"""Rows far weaker than the others, as rarely used ones have: their own error.

The first rounding of X counts most.  An entry is held to half a unit of
2^-24 of X scaled by 2^14 (|X| = 1), an error spread evenly over +-2^-25/2^14,
1/sqrt(3) of that in the root mean square.  It grows by at most 3.4445 an
iteration, and each iterate's own rounding adds to it:
sqrt(sum of 3.4445^(2k), k = 1..5) = 507 over five.  The products' roundings
add relative errors (2e-5 of the rows at most) and those of the Gram matrices'
entries, smaller ones; a factor of two covers them.
"""
from __future__ import annotations

import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315
ROUNDING = 2.0 ** -25 / 2.0 ** 14 / math.sqrt(3)
GROWTH = math.sqrt(sum(A ** (2 * k) for k in range(1, 6)))


def reference(u):
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        g = x @ x.t()
        x = A * x + B * (g @ x) + C * (g @ (g @ x))
    return x.t() if tall else x


@pytest.mark.parametrize("rows,cols", [(64, 64), (100, 900), (256, 256), (768, 768), (768, 2304), (2304, 768), (1031, 257)])
@pytest.mark.parametrize("grade", [1e-2, 1e-4, 1e-5, 1e-6, 1e-8])
def test_weak_rows(rows, cols, grade):
    u = torch.randn(rows, cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    half = rows // 2
    u[half:] *= grade
    out = torch.empty_like(u)
    with z.Muon(rows * cols, 1, [(0, rows, cols)]) as opt:
        opt.orthogonalize(u, out)
        opt.status()
    want = reference(u)
    err, size = (out.double() - want)[half:].norm().item(), want[half:].norm().item()
    entries = (rows - half) * cols
    assert err <= 2e-5 * size + 2 * ROUNDING * GROWTH * math.sqrt(entries)
    assert (out.double() - want).norm() <= 2e-5 * want.norm()
