"""Matrices stepped in one launch by clusters of one to eight blocks: larger
sides on both sides of every bound, slices of 64 to 256 columns, and last
blocks that hold few columns or none, against the definition in 64 bits.

Tolerances as in test_gpu_muon.py: 2e-5 of |X| after five iterations.  A
single direction (a side of one) is no looser: its one singular value keeps
its size.
"""
from __future__ import annotations

import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.gpu_util import Guarded
from tests.muon_tiles import small_blocks

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315
SIDES = [256, 257, 300, 384, 385, 513, 576, 577, 768, 769, 896, 897, 1025, 1152, 1153, 1344, 1345, 1536, 1537]


def reference(u):
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        g = x @ x.t()
        x = A * x + (B * g + C * (g @ g)) @ x
    return x.t() if tall else x


def view(flat, off, r, c):
    return torch.as_strided(flat, (r, c), (c, 1), flat.storage_offset() + off)


@pytest.mark.parametrize("side", SIDES)
@pytest.mark.parametrize("s", [1, 17, 100, 128])
@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalize(side, s, tall):
    r, c = (side, s) if tall else (s, side)
    assert small_blocks(r, c) == (1 if side <= 256 else 2 if side <= 384 else 4 if side <= 768 else 8 if side <= 1536 else 0)
    u = torch.randn(r, c, device="cuda", generator=torch.Generator(device="cuda").manual_seed(side * 7 + s))
    out = Guarded(r * c, torch.float32)
    with z.Muon(r * c, 1, [(0, r, c)]) as opt:
        opt.orthogonalize(u.view(-1), out.t)
        opt.status()
    want = reference(u)
    assert out.intact() and (out.t.view(r, c).double() - want).norm() <= 2e-5 * want.norm()


@pytest.mark.parametrize("world", [1, 9])
@pytest.mark.parametrize("tall", [False, True])
def test_step_of_all_sizes_in_one_list(world, tall):
    shapes = [(side, s) if tall else (s, side) for side in SIDES for s in (1, 17, 100, 128)]
    mats, n = [], 0
    for r, c in shapes:
        mats.append((n, r, c))
        n += r * c + 5
    g = torch.Generator(device="cuda").manual_seed(world)
    grads = [(1e-3 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(world)]
    params = [torch.full((n,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(world)]
    master, momentum = 0.02 * torch.randn(n, generator=g, device="cuda"), 5e-4 * torch.randn(n, generator=g, device="cuda")
    master0, momentum0 = master.clone(), momentum.clone()
    hp = z.MuonHparams()
    with z.Muon(n, world, mats, hp) as opt:
        opt.step(grads, params, master, momentum)
        opt.status()
    mean = sum(q.double() for q in grads) / world
    m = hp.momentum * momentum0.double() + (1 - hp.momentum) * mean
    u = hp.momentum * m + (1 - hp.momentum) * mean
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    for mt in mats:
        move = hp.lr * hp.update_scale * math.sqrt(max(mt[1:])) * reference(view(u, *mt))
        want = view(master0, *mt).double() * (1 - hp.lr * hp.weight_decay) - move
        # the sum of nine bf16 gradients and the momentum round in fp32 (12 of 2^-24), the master twice
        assert (view(master, *mt).double() - want).norm() <= 3e-5 * move.norm() + 2 * 2.0 ** -24 * want.norm()
        assert (view(momentum, *mt).double() - view(m, *mt)).norm() <= 12 * 2.0 ** -24 * view(m, *mt).norm()
        view(rest, *mt).fill_(False)
    low = master.to(torch.bfloat16)
    assert torch.equal(master[rest], master0[rest]) and torch.equal(momentum[rest], momentum0[rest])
    for q in params:
        assert torch.equal(q[~rest], low[~rest]) and (q[rest].float() == 5.0).all()
