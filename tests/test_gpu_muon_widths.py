"""Both widths of the tiled iteration: lists that the rule gives tiles of 256
columns (many matrices, or a large one) beside lists of 128, with remainders
in both sides, against the definition in 64 bits.

Tolerances as in test_gpu_muon.py (2e-5 of |X|): the kernels add up 128 of K
at a time, a wide tile's first two sums 256 each, with a relative loss of at
most 2e-6 a sum; a bf16 result adds its own rounding, 2^-8 of an entry.
"""
from __future__ import annotations

import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.gpu_util import Guarded
from tests.muon_tiles import tile_columns

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315
TOL = {torch.float32: 2e-5, torch.bfloat16: 2e-5 + 2.0 ** -8}

# name: (shapes, columns of a tile).  Lists of copies are one shape in many
# places, so that only a few of them are checked against 64 bits.
LISTS = {
    "narrow_wide_matrix": ([(300, 517)] * 5, 128),
    "narrow_tall_matrix": ([(517, 300)] * 5, 128),
    "wide_matrices": ([(300, 517)] * 120, 256),
    "tall_matrices": ([(517, 300)] * 120, 256),
    "long_sums": ([(257, 1031)] * 60 + [(1031, 257)] * 60, 256),
    "mixed": ([(129, 130), (255, 2050), (640, 200), (385, 385), (511, 513), (200, 1700), (1153, 131)] * 18, 256),
    "beside_small": ([(300, 517)] * 90 + [(64, 64), (40, 700), (1000, 128)], 256),
    "one_wide": ([(2305, 2567)], 256),
    "one_tall": ([(2567, 2305)], 256),
    "one_odd_square": ([(2311, 2311)], 256),
}


def sms() -> int:
    return torch.cuda.get_device_properties(0).multi_processor_count


def reference(u, steps=5, eps=1e-7):
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        g = x @ x.t()
        x = A * x + (B * g + C * (g @ g)) @ x
    return x.t() if tall else x


def view(flat, off, r, c, ld=None):
    return torch.as_strided(flat, (r, c), (ld or c, 1), flat.storage_offset() + off)


def place(shapes, gap=0):
    mats, at = [], 0
    for r, c in shapes:
        mats.append((at, r, c))
        at += r * c + gap
    return mats, at


def some(mats):
    """The first, the last and a few more of each shape."""
    by = {}
    for i, m in enumerate(mats):
        by.setdefault(m[1:], []).append(i)
    pick = set()
    for where in by.values():
        pick.update({where[0], where[-1], where[len(where) // 2], where[len(where) // 3]})
    return [mats[i] for i in sorted(pick)]


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("in_dtype,out_dtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)])
def test_against_the_definition(name, in_dtype, out_dtype):
    shapes, width = LISTS[name]
    assert tile_columns(shapes, sms()) == width
    mats, n = place(shapes, gap=3)
    u = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(len(name))).to(in_dtype)
    out, again = Guarded(n, out_dtype), torch.full((n,), 3.0, dtype=out_dtype, device="cuda")
    out.t.fill_(3.0)
    with z.Muon(n, 1, mats) as opt:
        opt.orthogonalize(u, out.t)
        opt.orthogonalize(u, again)
        opt.status()
    assert out.intact() and torch.equal(out.t, again)             # the same bits twice
    gaps = torch.ones(n, dtype=torch.bool, device="cuda")
    for m in mats:
        view(gaps, *m).fill_(False)
    assert (out.t[gaps].float() == 3.0).all()
    for m in some(mats):
        want = reference(view(u, *m))
        assert (view(out.t, *m).double() - want).norm() <= TOL[out_dtype] * want.norm(), m


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("shape", [(517, 300), (300, 517)])
def test_step_counts_with_wide_tiles(steps, shape):
    """The result lies in one of two regions by the count, in fp32 as the last product left it."""
    shapes = [shape] * 120
    assert tile_columns(shapes, sms()) == 256
    mats, n = place(shapes)
    u = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(steps))
    out = torch.empty_like(u)
    with z.Muon(n, 1, mats, z.MuonHparams(ns_steps=steps)) as opt:
        opt.orthogonalize(u, out)
        opt.status()
    for m in some(mats):
        want = reference(view(u, *m), steps)
        assert (view(out, *m).double() - want).norm() <= 2e-5 * want.norm()


def test_column_slices_with_wide_tiles():
    """The thirds of fused matrices, where they lie, in any order."""
    rows, cols, copies = 700, 260, 40
    mats = [(k * rows * 3 * cols + i * cols, rows, cols, 3 * cols) for k in range(copies) for i in (2, 0, 1)]
    n = copies * rows * 3 * cols
    assert tile_columns([(rows, cols)] * len(mats), sms()) == 256
    u = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).to(torch.bfloat16)
    out = torch.empty(n, device="cuda")
    with z.Muon(n, 1, mats) as opt:
        opt.orthogonalize(u, out)
        opt.status()
    for m in mats[:3] + mats[-3:]:
        want = reference(view(u, *m))
        assert (view(out, *m).double() - want).norm() <= 2e-5 * want.norm()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_stays_in_its_matrix_with_wide_tiles(bad):
    shapes = [(300, 517)] * 120
    mats, n = place(shapes)
    u = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    clean, out = torch.empty_like(u), torch.empty_like(u)
    with z.Muon(n, 1, mats) as opt:
        opt.orthogonalize(u, clean)
        u[mats[50][0] + 1234] = bad
        opt.orthogonalize(u, out)
        opt.status()
    assert torch.isnan(view(out, *mats[50])).all()
    for i, m in enumerate(mats):
        if i != 50:
            assert torch.equal(view(out, *m), view(clean, *m))


@pytest.mark.parametrize("world", [1, 3])
def test_step_with_wide_tiles(world):
    shapes = [(300, 517), (517, 300)] * 60
    assert tile_columns(shapes, sms()) == 256
    mats, n = place(shapes)
    g = torch.Generator(device="cuda").manual_seed(world)
    grads = [(1e-3 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(world)]
    params = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(world)]
    master, momentum = 0.02 * torch.randn(n, generator=g, device="cuda"), 5e-4 * torch.randn(n, generator=g, device="cuda")
    master0, momentum0 = master.clone(), momentum.clone()
    hp = z.MuonHparams()
    with z.Muon(n, world, mats, hp) as opt:
        opt.step(grads, params, master, momentum)
        opt.status()
    mean = sum(q.double() for q in grads) / world
    m = hp.momentum * momentum0.double() + (1 - hp.momentum) * mean
    u = hp.momentum * m + (1 - hp.momentum) * mean
    # four fp32 roundings of the momentum
    assert (momentum.double() - m).norm() <= 4 * 2.0 ** -24 * m.norm()
    for mt in some(mats):
        move = hp.lr * hp.update_scale * math.sqrt(max(mt[1:])) * reference(view(u, *mt))
        want = view(master0, *mt).double() * (1 - hp.lr * hp.weight_decay) - move
        err = (view(master, *mt).double() - want).norm()
        assert err <= 3e-5 * move.norm() + 2 * 2.0 ** -24 * want.norm()
    low = master.to(torch.bfloat16)
    assert all(torch.equal(q, low) for q in params)


@pytest.mark.parametrize("name", ["wide_matrices", "one_tall"])
def test_wide_tiles_on_part_of_the_sms(name):
    mats, n = place(LISTS[name][0])
    u = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    want, got = torch.empty_like(u), torch.empty_like(u)
    with z.Muon(n, 1, mats) as opt, z.SmPartition(16) as part:
        opt.orthogonalize(u, want)
        torch.cuda.synchronize()
        opt.orthogonalize(u, got, part.stream_a)
        opt.status(part.stream_a)
    assert torch.equal(want, got)


def test_a_wait_that_runs_out_with_wide_tiles():
    mats, n = place([(300, 517)] * 120)
    u = torch.randn(n, device="cuda")
    out = torch.empty_like(u)
    with z.Muon(n, 1, mats, z.MuonHparams(inject_wait_timeout=True)) as bad, z.Muon(n, 1, mats) as good:
        bad.orthogonalize(u, out)
        with pytest.raises(z.Zero1Error) as e:
            bad.status()
        assert e.value.code == -4 and "gave up" in str(e.value)
        good.orthogonalize(u, out)
        good.status()
    want = reference(view(u, *mats[0]))
    assert (view(out, *mats[0]).double() - want).norm() <= 2e-5 * want.norm()
