"""The matrix step and its orthogonalisation on the GPU against the definition
in 64 bits (numpy/torch fp64, elementary operations).

Tolerances, from the arithmetic and not from runs.  The iteration keeps 22
bits of every factor and sums 256 products at a time with a relative loss of
at most 2e-6, so one iteration's relative error is a few 1e-6; five compound
to below 2e-5 of |X| where the singular values are spread as in random
matrices.  Directions that start far below the largest grow by up to
3.4445^5 = 485, and the 2^-22 they start with grows with them: 485 * 2^-22 =
1.2e-4, so 2.5e-4 where a few directions carry almost all of the matrix.
An update moves the master by lr * scale * X, so its error there is the
same fraction of that, plus fp32 roundings of the master (2 * 2^-24).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.gpu_util import Guarded, bits_equal, f32, u16

pytestmark = pytest.mark.gpu

A, B, C = 3.4445, -4.7750, 2.0315
PLAIN, STRONG = 2e-5, 2.5e-4


def ref_orth(u: torch.Tensor, steps: int = 5, eps: float = 1e-7, abc=(A, B, C)) -> torch.Tensor:
    a, b, c = abc
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        g = x @ x.t()
        x = a * x + b * (g @ x) + c * (g @ (g @ x))
    return x.t() if tall else x


def rel(got: torch.Tensor, want: torch.Tensor) -> float:
    n = want.norm().item()
    return (got.double() - want).norm().item() / n if n else got.double().norm().item()


def view(flat, off, r, c, ld=None):
    return torch.as_strided(flat, (r, c), (ld or c, 1), flat.storage_offset() + off)


def run_orth(u: torch.Tensor, out_dtype=torch.float32, **hp) -> torch.Tensor:
    r, c = u.shape
    flat = u.contiguous().view(-1)
    out = Guarded(r * c, out_dtype)
    with z.Muon(r * c, 1, [(0, r, c)], z.MuonHparams(**hp)) as opt:
        opt.orthogonalize(flat, out.t)
        opt.status()
    assert out.intact()
    return out.t.view(r, c)


SIZES = [(1, 1), (1, 2), (2, 1), (1, 300), (300, 1), (3, 5), (8, 8), (17, 33), (63, 64), (64, 65), (127, 129), (128, 128),
         (129, 127), (200, 64), (255, 257), (256, 256), (257, 255), (64, 1000), (1000, 64), (130, 513), (300, 1200),
         (385, 770), (1031, 257), (520, 520), (768, 768), (1, 70000), (40, 20001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_random(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * 100003 + cols)
    u = torch.randn(rows, cols, generator=g, device="cuda").mul_(1e-3).to(dtype)
    assert rel(run_orth(u), ref_orth(u)) <= PLAIN


@pytest.mark.parametrize("shapes", [[(150, 4000)], [(4000, 150)], [(257, 3001)], [(513, 2050), (2050, 140)],
                                    [(200, 9000), (300, 300), (1030, 129), (40, 50), (17, 2000)]])
def test_long_sums_and_mixed_lists(shapes):
    """Gram matrices formed in slices of K, beside matrices that are not, and
    beside small ones; the same bits twice."""
    mats, at = [], 0
    for r, c in shapes:
        mats.append((at, r, c))
        at += r * c
    u = torch.randn(at, generator=torch.Generator(device="cuda").manual_seed(at), device="cuda")
    out, again = torch.empty_like(u), torch.empty_like(u)
    with z.Muon(at, 1, mats) as opt:
        opt.orthogonalize(u, out)
        opt.orthogonalize(u, again)
        opt.status()
    assert torch.equal(out, again)
    assert max(rel(view(out, *m), ref_orth(view(u, *m))) for m in mats) <= PLAIN


@pytest.mark.parametrize("rows,cols", [(64, 64), (256, 256), (300, 1100), (900, 130)])
@pytest.mark.parametrize("kind", ["decay", "strong", "rank1"])
def test_orthogonalize_uneven_spectra(rows, cols, kind):
    g = torch.Generator(device="cuda").manual_seed(5)
    k = min(rows, cols)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)

    if kind == "decay":
        p, q = torch.linalg.qr(randn(rows, k))[0], torch.linalg.qr(randn(cols, k))[0]
        u = (p * torch.logspace(0, -4, k, device="cuda", dtype=torch.float64)) @ q.t()
    elif kind == "strong":
        u = randn(rows, 4) @ randn(4, cols) + 1e-4 * randn(rows, cols)
    else:
        u = randn(rows, 1) @ randn(1, cols)
    u = u.float()
    assert rel(run_orth(u), ref_orth(u)) <= STRONG


def test_singular_values_come_near_one():
    g = torch.Generator(device="cuda").manual_seed(9)
    s = torch.linalg.svdvals(run_orth(torch.randn(200, 330, generator=g, device="cuda")).double())
    assert s.min() > 0.6 and s.max() < 1.3


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_step_counts_and_coefficients(steps):
    g = torch.Generator(device="cuda").manual_seed(steps)
    u = torch.randn(150, 310, generator=g, device="cuda")
    assert rel(run_orth(u, ns_steps=steps), ref_orth(u, steps)) <= PLAIN
    abc = (1.875, -1.25, 0.375)     # the quintic that converges to one
    got = run_orth(u, ns_steps=steps, ns_a=abc[0], ns_b=abc[1], ns_c=abc[2])
    assert rel(got, ref_orth(u, steps, abc=abc)) <= PLAIN


@pytest.mark.parametrize("scale", [1e-18, 1e-9, 1.0, 1e9, 1e18])
def test_scale_of_the_input_does_not_matter(scale):
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.randn(100, 120, generator=g, device="cuda") * scale
    assert rel(run_orth(u, eps=1e-15), ref_orth(u, eps=1e-15)) <= PLAIN


def test_zero_matrix_stays_zero():
    assert run_orth(torch.zeros(130, 70, device="cuda")).abs().max().item() == 0.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_spoils_its_own_matrix_only(bad):
    mats = [(0, 130, 140), (130 * 140, 300, 64), (130 * 140 + 300 * 64, 64, 64)]
    n = 130 * 140 + 300 * 64 + 64 * 64
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(n, generator=g, device="cuda")
    clean, out = torch.empty_like(u), torch.empty_like(u)
    with z.Muon(n, 1, mats) as opt:
        opt.orthogonalize(u, clean)
        u[mats[1][0] + 77] = bad
        opt.orthogonalize(u, out)
        opt.status()
    assert torch.isnan(view(out, *mats[1])).all()
    for m in (mats[0], mats[2]):
        assert torch.equal(view(out, *m), view(clean, *m))


@pytest.mark.parametrize("in_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_flat_buffer_strides_offsets_and_untouched_entries(in_dtype, out_dtype):
    """Interleaved column slices, padded rows, odd offsets, any order; what no
    matrix covers keeps its bits."""
    qkv = [(8 + 96 * i, 50, 96, 288) for i in range(3)]              # aligned slices of one 50 x 288 matrix
    at = 8 + 50 * 288
    mats = [(at + 3, 33, 21, 29), qkv[2], qkv[0], (at + 3 + 33 * 29 + 5, 1, 200), qkv[1],
            (at + 3 + 33 * 29 + 400, 70, 40, 48)]
    n = at + 3 + 33 * 29 + 400 + 70 * 48 + 11
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(n, generator=g, device="cuda").to(in_dtype)
    out = Guarded(n, out_dtype)
    out.t.fill_(3.0)
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    with z.Muon(n, 1, mats) as opt:
        assert opt.layout()[0] == sum(m[1] * m[2] for m in mats)
        opt.orthogonalize(u, out.t)
        opt.status()
    assert out.intact()
    for m in mats:
        want = ref_orth(view(u, *m))
        tol = PLAIN if out_dtype == torch.float32 else PLAIN + 2.0 ** -8
        assert rel(view(out.t, *m), want) <= tol
        view(mask, *m).fill_(False)
    assert (out.t[mask].float() == 3.0).all()


def test_in_place_and_between_types():
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.randn(90 * 60, generator=g, device="cuda")
    with z.Muon(90 * 60, 1, [(0, 90, 60)]) as opt:
        want = torch.empty_like(u)
        opt.orthogonalize(u, want)
        low = torch.empty_like(u, dtype=torch.bfloat16)
        opt.orthogonalize(u, low)
        opt.orthogonalize(u, u)
        opt.status()
    assert torch.equal(u, want)
    assert torch.equal(low, want.to(torch.bfloat16))


def test_many_matrices_of_many_shapes():
    rng = np.random.default_rng(7)
    mats, at = [], 0
    for _ in range(300):
        r, c = (int(math.exp(rng.uniform(0, math.log(200)))) for _ in range(2))
        mats.append((at, r, c))
        at += r * c
    g = torch.Generator(device="cuda").manual_seed(8)
    u = torch.randn(at, generator=g, device="cuda")
    out = torch.empty_like(u)
    with z.Muon(at, 1, mats) as opt:
        opt.orthogonalize(u, out)
        opt.status()
    assert max(rel(view(out, *m), ref_orth(view(u, *m))) for m in mats) <= PLAIN


# ----------------------------------------------------------------- step

def problem(shapes, world, seed=0):
    mats, at = [], 0
    for r, c in shapes:
        mats.append((at, r, c))
        at += r * c
    n = at + 24                                   # entries no matrix covers
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(s):
        return torch.randn(n, generator=g, device="cuda") * s

    grads = [Guarded(n, torch.bfloat16) for _ in range(world)]
    params = [Guarded(n, torch.bfloat16) for _ in range(world)]
    for q in grads:
        q.t.copy_(randn(1e-3))
    for q in params:
        q.t.fill_(5.0)
    master, momentum = Guarded(n, torch.float32), Guarded(n, torch.float32)
    master.t.copy_(randn(0.02))
    momentum.t.copy_(randn(5e-4))
    return mats, n, grads, params, master, momentum


def check_step(mats, n, grads, params, master, momentum, hp, master0, momentum0):
    gm = torch.stack([q.t.double() for q in grads]).mean(0)
    m = hp.momentum * momentum0.double() + (1 - hp.momentum) * gm
    u = hp.momentum * m + (1 - hp.momentum) * gm if hp.nesterov else m
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    for mt in mats:
        _, r, c = mt
        factor = math.sqrt(max(r, c)) if hp.scale_rule == z.SCALE_RMS else math.sqrt(max(1.0, r / c))
        move = hp.lr * hp.update_scale * factor * ref_orth(view(u, *mt), hp.ns_steps, hp.eps)
        want = view(master0, *mt).double() * (1 - hp.lr * hp.weight_decay) - move
        # the momentum's own fp32 roundings (4 of 2^-24) enter U, and X with at most the same relative size
        err = (view(master.t, *mt).double() - want).norm().item()
        assert err <= PLAIN * 1.5 * move.norm().item() + 2 * 2.0 ** -24 * want.norm().item() + 1e-12
        assert rel(view(momentum.t, *mt), view(m, *mt)) <= 4 * 2.0 ** -24
        view(rest, *mt).fill_(False)
    low = master.t.to(torch.bfloat16)
    for q in params:
        assert torch.equal(q.t[~rest], low[~rest]) and (q.t[rest].float() == 5.0).all() and q.intact()
    assert torch.equal(master.t[rest], master0[rest]) and torch.equal(momentum.t[rest], momentum0[rest])
    assert master.intact() and momentum.intact() and all(q.intact() for q in grads)


@pytest.mark.parametrize("world", [1, 2, 3, 8, 9, 65])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(world, nesterov):
    mats, n, grads, params, master, momentum = problem([(64, 64), (96, 40), (31, 77), (200, 264), (1, 9)], world, world)
    hp = z.MuonHparams(nesterov=nesterov, scale_rule=z.SCALE_SPECTRAL if world == 3 else z.SCALE_RMS)
    a, b = master.t.clone(), momentum.t.clone()
    with z.Muon(n, world, mats, hp) as opt:
        opt.step([q.t for q in grads], [q.t for q in params], master.t, momentum.t)
        opt.status()
    check_step(mats, n, grads, params, master, momentum, hp, a, b)


def test_steps_follow_on_another_stream_with_a_new_rate():
    mats, n, grads, params, master, momentum = problem([(130, 150), (150, 130)], 2, 11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hp = z.MuonHparams()
    with z.Muon(n, 2, mats, hp) as opt:
        for lr in (1e-3, 5e-4, 0.0):
            opt.set_lr(lr)
            hp.lr = lr
            a, b = master.t.clone(), momentum.t.clone()
            side.wait_stream(torch.cuda.current_stream())
            opt.step(z.PtrTable([q.t for q in grads]), z.PtrTable([q.t for q in params]), master.t, momentum.t, side)
            opt.status(side)
            check_step(mats, n, grads, params, master, momentum, hp, a, b)


def test_step_is_deterministic_and_can_be_captured():
    def run(graph):
        mats, n, grads, params, master, momentum = problem([(300, 140), (64, 500), (64, 64)], 2, 21)
        args = ([q.t for q in grads], [q.t for q in params], master.t, momentum.t)
        with z.Muon(n, 2, mats) as opt:
            opt.step(*args, torch.cuda.current_stream())
            if graph:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    opt.step(*args, torch.cuda.current_stream())
                g.replay()
                g.replay()
            else:
                opt.step(*args, torch.cuda.current_stream())
                opt.step(*args, torch.cuda.current_stream())
            torch.cuda.synchronize()
            opt.status()
        return f32(master.t), f32(momentum.t), u16(params[1].t)
    first, second, third = run(False), run(False), run(True)
    for other in (second, third):
        assert bits_equal(first[0], other[0]) and bits_equal(first[1], other[1])
        assert np.array_equal(first[2], other[2])


def test_runs_on_part_of_the_sms():
    """The iteration does not need its blocks to be resident together."""
    u = torch.randn(700 * 900, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    want, got = torch.empty_like(u), torch.empty_like(u)
    with z.Muon(u.numel(), 1, [(0, 700, 900)]) as opt:
        opt.orthogonalize(u, want)
        torch.cuda.synchronize()
        with z.SmPartition(16) as part:
            opt.orthogonalize(u, got, part.stream_a)
            opt.status(part.stream_a)
    assert torch.equal(want, got)


def test_beside_adamw_for_the_vectors():
    """Matrices first in the flat buffers, then the vectors, which an AdamW
    handle steps through offset pointers; neither touches the other's."""
    mats, n, grads, params, master, momentum = problem([(64, 96), (96, 64)], 2, 31)
    vec = n - 24                                   # a multiple of 8: 16-byte aligned in bf16
    assert vec % 8 == 0
    a, b = master.t.clone(), momentum.t.clone()
    hp = z.MuonHparams()
    with z.Muon(n, 2, mats, hp) as opt, z.Zero1(24, 2, z.Hparams(max_norm=0.0)) as adam:
        adam.set_state(master.t[vec:])
        opt.step([q.t for q in grads], [q.t for q in params], master.t, momentum.t)
        for q in params:
            assert (q.t[vec:].float() == 5.0).all()
        check_step(mats, n, grads, params, master, momentum, hp, a, b)
        before = [u16(q.t[:vec]) for q in params]
        adam.step([q.t[vec:] for q in grads], [q.t[vec:] for q in params])
        m2 = torch.empty(24, device="cuda")
        adam.get_state(m2)
        torch.cuda.synchronize()
    for q, old in zip(params, before):
        assert np.array_equal(u16(q.t[:vec]), old)
        assert torch.equal(q.t[vec:], m2.to(torch.bfloat16))


def test_refusals():
    x = torch.zeros(64 * 64 + 8, device="cuda")
    h = torch.zeros(64 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    with z.Muon(64 * 64, 2, [(0, 64, 64)]) as opt:
        for args in (([h[1:], h], [h, h], x, x), ([h, h], [h, h[1:]], x, x), ([h, h], [h, h], x[1:], x)):
            with pytest.raises(z.Zero1Error) as e:
                opt.step(*args)
            assert e.value.code == -2
        for args in (([h], [h, h], x, x), ([h, h], [h, h], h, x), ([h, h], [h, h], x, x[:100]), ([x, x], [h, h], x, x),
                     ([h, h], [h, h], x.cpu(), x)):
            with pytest.raises(z.Zero1ArgumentError):
                opt.step(*args)
        with pytest.raises(z.Zero1Error) as e:
            opt.orthogonalize(x[1:], x)
        assert e.value.code == -2
        with pytest.raises(z.Zero1Error):
            z.zero1_muon_orthogonalize(opt.handle, x, 7, x, z.DTYPE_F32)
        with pytest.raises(z.Zero1ArgumentError):
            opt.orthogonalize(x.half(), x)
        with pytest.raises(z.Zero1Error):
            opt.set_lr(float("nan"))
        opt.status()
    with pytest.raises(z.Zero1Error):
        z.zero1_muon_step(opt.handle or 0xDEAD0000, [h, h], [h, h], x, x)


def test_a_wait_that_runs_out_is_reported():
    """No tile is ever drawn: every wait of the iteration gives up after its
    limit, the call ends, the status says so for this handle and no other,
    and the device goes on."""
    u = torch.randn(300 * 200, device="cuda")
    out = torch.empty_like(u)
    with z.Muon(u.numel(), 1, [(0, 300, 200)], z.MuonHparams(inject_wait_timeout=True)) as bad, \
            z.Muon(u.numel(), 1, [(0, 300, 200)]) as good:
        bad.orthogonalize(u, out)
        with pytest.raises(z.Zero1Error) as e:
            bad.status()
        assert e.value.code == -4 and "gave up" in str(e.value)
        good.orthogonalize(u, out)
        good.status()
        assert rel(view(out, 0, 300, 200), ref_orth(view(u, 0, 300, 200))) <= PLAIN
        with pytest.raises(z.Zero1Error):
            bad.status()


def test_offsets_past_32_bits():
    """A large and a small matrix that lie beyond 2^32 entries of their buffer."""
    at = (1 << 32) + 24
    mats = [(at, 200, 150), (at + 200 * 150, 40, 64)]
    n = at + 200 * 150 + 40 * 64
    flat = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    u = torch.randn(n - at, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(torch.bfloat16)
    flat[at:] = u
    with z.Muon(n, 1, mats) as opt:
        opt.orthogonalize(flat, flat)
        opt.status()
    for off, r, c in mats:
        got, want = view(flat, off, r, c), ref_orth(view(u, off - at, r, c))
        assert rel(got, want) <= PLAIN + 2.0 ** -8
    assert not flat[:4096].any() and not flat[at - 4096:at].any()
    del flat
    torch.cuda.empty_cache()


def test_a_refused_allocation_leaves_no_error_behind():
    """Eight matrices of 65,536 x 65,536 need half a terabyte: creation says so,
    and the calls after it on the same thread are judged by their own launches."""
    side = 65536
    with pytest.raises(z.Zero1Error) as e:
        z.Muon(8 * side * side, 1, [(i * side * side, side, side) for i in range(8)])
    assert e.value.code == -3, e.value
    x = torch.randn(16, 300, device="cuda")
    y, mean, rstd, gamma = torch.empty_like(x), torch.empty(16, device="cuda"), torch.empty(16, device="cuda"), torch.ones(300, device="cuda")
    z.zero1_layernorm_forward(16, 300, z.DTYPE_F32, x, 300, gamma, None, 1e-5, y, 300, mean, rstd)
    assert rel(y, torch.nn.functional.layer_norm(x.double(), (300,), eps=1e-5)) < 1e-6
    u = torch.randn(130, 140, device="cuda")
    assert rel(run_orth(u), ref_orth(u)) < PLAIN
