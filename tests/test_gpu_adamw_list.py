"""AdamW over many tensors on the GPU: bit for bit the written formulas, near
them in 64 bits, and what the 8-bit moments promise."""
import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import adamw_plain as ap

pytestmark = pytest.mark.gpu

SIZES = [768, 0, 1, 255, 256, 257, 2049, 64 * 63, 5000, 3]
DT = {"bf16": (torch.bfloat16, z.DTYPE_BF16), "f32": (torch.float32, z.DTYPE_F32)}


class Case:
    """A list of tensors with its state, and the plain step of the same."""

    def __init__(self, sizes, param="bf16", grad="bf16", bits=32, hp=None, decays=None, decay_first=False, seed=5,
                 offset=0, t=0, scale=1e-2):
        self.hp = hp or z.Hparams(max_norm=0.05)
        self.sizes, self.bits, self.seed, self.first = sizes, bits, seed, decay_first
        self.starts, self.n = ap.starts(sizes)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.scale = gen, scale
        self.dp, self.dg = DT[param][0], DT[grad][0]
        # tensors `offset` entries past a 16-byte boundary, each in memory of its own
        self.params = [torch.empty(n + offset + 8, dtype=self.dp, device="cuda")[offset:offset + n] for n in sizes]
        self.grads = [torch.empty(n + offset + 8, dtype=self.dg, device="cuda")[offset:offset + n] for n in sizes]
        flat = torch.randn(self.n, generator=gen, device="cuda") * 0.02
        for p, a in zip(self.params, self.starts):
            p.copy_(flat[a:a + p.numel()])
        self.master = flat.clone() if param == "bf16" else None
        self.mask = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        self.decays = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        for i, (a, n) in enumerate(zip(self.starts, sizes)):
            self.mask[a:a + n] = True
            self.decays[a:a + n] = True if decays is None else bool(decays[i])
        kind = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = torch.zeros(self.n, dtype=kind, device="cuda"), torch.zeros(self.n, dtype=kind, device="cuda")
        self.scales = None if bits == 32 else torch.zeros(self.n // 128, device="cuda")
        self.opt = z.AdamW(sizes, self.hp, z.AdamWOptions(state_bits=bits, param_dtype=DT[param][1],
                                                          grad_dtype=DT[grad][1], decay_before_update=decay_first,
                                                          seed=seed), decays)
        assert (self.opt.entries, self.opt.starts) == (self.n, self.starts)
        self.t = t
        self.opt.set_steps(t)
        # what lies between tensors must stay
        fill = 77 if bits == 8 else 3.25
        for x in (self.m, self.v) + ((self.master,) if self.master is not None else ()):
            x[~self.mask] = fill if x.dtype == self.m.dtype else 3.25

    def draw(self):
        for g in self.grads:
            g.copy_(torch.randn(g.numel(), generator=self.gen, device="cuda") * self.scale
                    * torch.exp(2 * torch.randn(g.numel(), generator=self.gen, device="cuda")))

    def flat(self, tensors):
        out = torch.zeros(self.n, device="cuda")
        for x, a in zip(tensors, self.starts):
            out[a:a + x.numel()] = x.float()
        return out

    def moments(self):
        if self.bits == 32:
            return self.m * self.mask, self.v * self.mask
        m, r = ap.decode(self.m, self.v, self.scales.view(-1, 2))
        return torch.where(self.mask, m, 0.), torch.where(self.mask, r * r, 0.)

    def run(self, stream=None):
        self.opt.step(self.grads, self.params, self.master, self.m, self.v, self.scales, stream)

    def plain(self):
        """What the next step makes of the present tensors and state."""
        self.t += 1
        g = self.flat(self.grads)
        w = torch.where(self.mask, self.master, 0.) if self.master is not None else self.flat(self.params)
        m, v = self.moments()
        clip = None
        if self.hp.max_norm > 0:
            norm = torch.cat([x.double() for x in self.grads]).square().sum().sqrt()
            clip = torch.clamp(self.hp.max_norm / norm, max=1.0).float()
        w, m, v = ap.step(g, w, m, v, self.hp, self.t, self.decays, clip, self.first)
        want = {"w": w, "clip": clip}
        if self.bits == 32:
            return want | {"m": m, "v": v}
        a, b = ap.dither(self.n, self.seed, self.t, "cuda")
        km, sm = ap.encode(torch.where(self.mask, m, 0.), ap.M_TOP, 3, a, False)
        kr, sr = ap.encode(torch.where(self.mask, v.sqrt(), 0.), ap.R_TOP, 4, b, True)
        km = torch.where(m < 0, km + 128, km)
        return want | {"km": km, "kr": kr, "scales": torch.stack([sm, sr], 1)}

    def check(self, want):
        keep = lambda x: x[self.mask]  # noqa: E731
        same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))  # noqa: E731
        if self.master is not None:
            assert same(keep(self.master), keep(want["w"]))
            assert bool((self.master[~self.mask] == 3.25).all())
        for p, a in zip(self.params, self.starts):
            assert torch.equal(p, want["w"][a:a + p.numel()].to(self.dp))
        if self.bits == 32:
            assert same(keep(self.m), keep(want["m"])) and same(keep(self.v), keep(want["v"]))
            assert bool((self.m[~self.mask] == 3.25).all()) and bool((self.v[~self.mask] == 3.25).all())
        else:
            assert torch.equal(keep(self.m).long(), keep(want["km"]))
            assert torch.equal(keep(self.v).long(), keep(want["kr"]))
            assert torch.equal(self.scales.view(-1, 2), want["scales"])
            assert bool((self.m[~self.mask] == 77).all()) and bool((self.v[~self.mask] == 77).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps_are_the_written_formulas_bit_for_bit(param, grad, bits, offset):
    c = Case(SIZES, param, grad, bits, offset=offset)
    for _ in range(4):
        c.draw()
        want = c.plain()
        c.run()
        c.check(want)
    assert c.opt.steps() == 4
    c.opt.close()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hp,first", [(z.Hparams(max_norm=0.0), False), (z.Hparams(max_norm=1e9), True),
                                      (z.Hparams(beta1=0.0, beta2=0.0, max_norm=0.0), False),
                                      (z.Hparams(beta2=0.999, weight_decay=0.0, eps=1e-6, max_norm=0.01), True),
                                      (z.Hparams(lr=0.0, max_norm=1.0), False)])
def test_variants(hp, first, bits):
    c = Case([4096, 300, 257], bits=bits, hp=hp, decays=[1, 0, 1], decay_first=first, t=7)
    for _ in range(3):
        c.draw()
        want = c.plain()
        c.run()
        c.check(want)
    if hp.max_norm > 0:
        norm, clip = c.opt.grad_norm()
        assert clip == float(want["clip"])
        exact = float(torch.cat([g.double() for g in c.grads]).square().sum().sqrt())
        # 32 bits twice: 2^-47 a square and an addition, fewer than 2^6 of them a thread, then fp64
        assert abs(norm - exact) <= exact * 2.0 ** -40


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_take_several_launches(bits):
    """2,100 tensors: more pointers than one launch holds; some at the end are empty."""
    sizes = [(i * 37) % 400 for i in range(2095)] + [0] * 5
    c = Case(sizes, bits=bits)
    for _ in range(2):
        c.draw()
        want = c.plain()
        c.run()
        c.check(want)
    c = Case([300] + [0] * 2000, bits=bits)   # nothing left for the last launch
    c.draw()
    want = c.plain()
    c.run()
    c.check(want)
    assert c.opt.steps() == 1


@pytest.mark.parametrize("count", [32, 33, 256, 257])
def test_at_the_bounds_of_a_launch(count):
    c = Case([40 + i % 7 for i in range(count)], bits=8)
    c.draw()
    want = c.plain()
    c.run()
    c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_near_64_bits(bits):
    """One step against 64 bits from the same state.  Each of m, v and the
    update is at most six roundings of 2^-24 (three of scalars, three of
    operations; v one more from sqrt and its square in 8 bits, u two more), of
    terms that do not exceed |beta1 m| + |(1-beta1) g|, v and |u|."""
    c = Case([20000, 333], bits=bits, hp=z.Hparams(max_norm=0.3), t=10)
    for _ in range(3):
        c.draw()
        c.run()
    c.t += 3
    c.draw()
    hp, t = c.hp, c.t + 1
    g = c.flat(c.grads).double()
    g = g * min(1.0, hp.max_norm / float(g.norm()))
    m, v = (x.double() for x in c.moments())
    w = torch.where(c.mask, c.master, 0.).double()
    c.run()
    terms = (hp.beta1 * m).abs() + ((1 - hp.beta1) * g).abs()
    m = hp.beta1 * m + (1 - hp.beta1) * g
    v = hp.beta2 * v + (1 - hp.beta2) * g * g
    size, keep = ap.scalars(hp, t)
    u = size * m / (v.sqrt() + hp.eps)
    du = size * terms / (v.sqrt() + hp.eps)
    want = (w - u) * keep
    e = 2.0 ** -24
    assert bool(((c.master.double() - want).abs() <= 16 * e * (w.abs() + du) )[c.mask].all())
    low = torch.cat([p.double() for p in c.params])
    full = torch.cat([c.master[a:a + n] for a, n in zip(c.starts, c.sizes)]).double()
    assert bool(((low - full).abs() <= full.abs() * 2.0 ** -8).all())
    got_m, got_v = c.moments()
    if bits == 32:
        assert bool(((got_m.double() - m).abs() <= 8 * e * terms).all())
        assert bool(((got_v.double() - v).abs() <= 10 * e * v).all())
    else:
        # a code's width: 2^-3 (m) and 2^-4 (sqrt v) of value + one unit of the block, and a code never below
        # the first for sqrt v > 0
        um, ur = (c.scales.view(-1, 2)[:, i].double().repeat_interleave(256) for i in (0, 1))
        assert bool(((got_m.double() - m).abs() <= (m.abs() + um) * (2.0 ** -3 + 1e-4)).all())
        r = v.sqrt()
        assert bool(((got_v.double().sqrt() - r).abs() <= (r + ur) * (2.0 ** -4 + 1e-4)).all())


def test_moments_are_what_the_codes_stand_for():
    c = Case(SIZES, bits=8)
    for _ in range(3):
        c.draw()
        c.run()
    mo, vo = torch.full((c.n,), 9.0, device="cuda"), torch.full((c.n,), 9.0, device="cuda")
    c.opt.moments(c.m, c.v, c.scales, mo, vo)
    m, v = c.moments()
    assert torch.equal(mo[c.mask], m[c.mask]) and torch.equal(vo[c.mask], v[c.mask])
    assert bool((mo[~c.mask] == 9).all()) and bool((vo[~c.mask] == 9).all())
    again = torch.zeros_like(mo)
    c.opt.moments(c.m, c.v, c.scales, None, again)
    assert torch.equal(again[c.mask], v[c.mask])


def test_eight_bit_means_are_unbiased():
    """Without gradients v decays by beta2 a step, 5%: less than half a code's
    width, so rounding to nearest would hold it.  Over 65,536 entries of like
    size the mean of v after 40 steps is 0.95^40 of the first: a step's
    rounding is unbiased in sqrt(v) with a variance of at most (2^-4 r)^2 / 4,
    which adds at most 2^-10 of v a step (in all 4%), and entries' random
    walks average out to 1e-3."""
    hp = z.Hparams(max_norm=0.0, lr=0.0)
    c = Case([65536], bits=8, hp=hp)
    c.grads[0].copy_(torch.randn(65536, generator=c.gen, device="cuda").sign() * (0.5 + torch.rand(65536, device="cuda")))
    c.run()
    m0, v0 = (x.double() for x in c.moments())
    c.grads[0].zero_()
    for _ in range(40):
        c.run()
    m, v = (x.double() for x in c.moments())
    ratio = float(v.mean() / v0.mean()) / hp.beta2 ** 40
    assert 0.99 <= ratio <= 1.05, ratio
    # m: (2^-3)^2 / 4 a step of its square at most, 40 steps: 40% an entry, 0.16% over 65,536; six times that
    ratio = float((m * m0.sign()).mean() / m0.abs().mean()) / hp.beta1 ** 40
    assert abs(ratio - 1) <= 0.01, ratio


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_is_not_finite_stays_in_its_place(bits, bad):
    """Without clipping: in 32 bits the entry alone, in 8 bits its block's moments."""
    c = Case([1024, 600], bits=bits, hp=z.Hparams(max_norm=0.0))
    c.draw()
    c.grads[0][300] = bad
    want = c.plain()
    c.run()
    p = torch.cat([x.float() for x in c.params])
    assert bool(p[300].isnan()) and int(p.isnan().sum()) == 1
    m, v = c.moments()
    if bits == 32:
        assert int((~m.isfinite()).sum()) == 1 and int((~v.isfinite()).sum()) == 1
    else:
        assert torch.equal(m.isnan().nonzero().view(-1), torch.arange(256, 512, device="cuda"))
        assert torch.equal(v.isnan().nonzero().view(-1), torch.arange(256, 512, device="cuda"))
        assert torch.equal(c.m.long()[c.mask], want["km"][c.mask])


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_a_norm_that_is_not_finite(bits):
    c = Case([512], bits=bits, hp=z.Hparams(max_norm=1.0))
    c.draw()
    c.grads[0][3] = math.nan
    c.run()
    assert bool(c.params[0].isnan().all()) and math.isnan(c.opt.grad_norm()[0])
    c = Case([512], bits=bits, hp=z.Hparams(max_norm=1.0))
    c.draw()
    c.grads[0][3] = math.inf
    c.run()
    assert c.opt.grad_norm() == (math.inf, 0.0)
    assert c.params[0].isnan().nonzero().view(-1).tolist() == [3]


@pytest.mark.parametrize("size", [1e-18, 1e-25, 1e25, 1e-3])
def test_norm_of_extreme_gradients(size):
    """Squares that leave fp32's range are summed in fp64."""
    c = Case([3000, 257], "f32", "f32", hp=z.Hparams(max_norm=1.0), scale=size)
    c.draw()
    c.run()
    exact = float(torch.cat([g.double() for g in c.grads]).square().sum().sqrt())
    norm, clip = c.opt.grad_norm()
    assert abs(norm - exact) <= exact * 2.0 ** -40
    assert clip == (1.0 if exact <= 1 else float(torch.tensor(1.0 / exact, dtype=torch.float64).float()))


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[512], [256 * 40], [256 * 31 + 5, 700]])
@pytest.mark.parametrize("at", [0, 3, 300, 511])
def test_norm_with_one_extreme_entry(sizes, at, grad):
    """One entry of 2^62 among ordinary ones: its thread's sum is taken again, of the same entries."""
    c = Case(sizes, "f32", grad, hp=z.Hparams(max_norm=1.0))
    c.draw()
    c.grads[0][at] = 2.0 ** 62
    c.run()
    exact = float(torch.cat([g.double() for g in c.grads]).square().sum().sqrt())
    assert abs(c.opt.grad_norm()[0] - exact) <= exact * 2.0 ** -40
    # and the others still count
    c.grads[0].mul_(0)
    c.grads[0][:5] = 3.0
    c.grads[0][at] = 2.0 ** -60
    c.run()
    exact = float(torch.cat([g.double() for g in c.grads]).square().sum().sqrt())
    assert abs(c.opt.grad_norm()[0] - exact) <= exact * 2.0 ** -40


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 0.0, 1e-30])
def test_entries_of_every_size(bits, eps):
    """Gradients of 1e-30 to 1e18, zeros among them: roots and quotients near
    the ends of fp32's range and away from it round the same way."""
    c = Case([4096, 300], "f32", "f32", bits, hp=z.Hparams(max_norm=0.0, eps=eps))
    for turn in range(4):
        for g in c.grads:
            n = g.numel()
            size = torch.exp(math.log(10) * (48 * torch.rand(n, generator=c.gen, device="cuda") - 30))
            g.copy_(torch.randn(n, generator=c.gen, device="cuda") * size)
            g[torch.rand(n, generator=c.gen, device="cuda") < 0.1] = 0.0
            if turn % 2 == 0:    # rows of one size, as real ones are
                g[:n // 2] = torch.randn(n // 2, generator=c.gen, device="cuda") * 10.0 ** (turn * 9 - 25)
        want = c.plain()
        c.run()
        fine = want["w"].isfinite()          # 0 / 0 without eps is NaN on both sides
        assert torch.equal(c.flat(c.params)[fine], (want["w"] * c.mask)[fine])
        assert torch.equal(c.flat(c.params).isnan(), (want["w"].isnan() & c.mask))
        for p in c.params:
            p.nan_to_num_(0.0)
        if bits == 32:
            assert torch.equal(c.m[c.mask], want["m"][c.mask]) and torch.equal(c.v[c.mask], want["v"][c.mask])
        else:
            assert torch.equal(c.m.long()[c.mask] & 127, want["km"][c.mask] & 127)
            assert torch.equal(c.v.long()[c.mask], want["kr"][c.mask])


def test_zeros_and_blocks_below_the_least_scale():
    c = Case([512, 256], bits=8, hp=z.Hparams(max_norm=0.0))
    c.grads[0].zero_()
    c.grads[1].fill_(1e-36)
    want = c.plain()
    c.run()
    c.check(want)
    m, v = c.moments()
    assert not bool(m.any()) and not bool(v.any()) and not bool(c.scales.any())


def test_a_captured_step_replays_as_the_next_one():
    a, b = Case(SIZES, bits=8), Case(SIZES, bits=8)
    a.draw()
    for x, y in zip(b.grads, a.grads):
        x.copy_(y)
    for _ in range(5):
        a.run()
    a.opt.set_lr(5e-4)
    a.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            b.run(torch.cuda.current_stream())
        for _ in range(4):
            graph.replay()
        b.opt.set_lr(5e-4, s)
        graph.replay()
    s.synchronize()
    torch.cuda.synchronize()
    assert a.opt.steps() == b.opt.steps() == 6
    for x, y in zip([a.master, a.m, a.v, a.scales] + a.params, [b.master, b.m, b.v, b.scales] + b.params):
        assert torch.equal(x, y)


def test_places_past_32_bits():
    """A tensor of 2^32 + 1,000 entries with 8-bit moments: the entries around
    and past 2^32, whose random bits take the upper half of their place."""
    n, hp = (1 << 32) + 1000, z.Hparams(max_norm=0.0)
    entries = -(-n // 256) * 256
    first = (1 << 32) - 512
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    param = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    master = torch.zeros(entries, device="cuda")
    m, v = (torch.zeros(entries, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = torch.zeros(entries // 128, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    grad[first:] = torch.randn(n - first, generator=gen, device="cuda").bfloat16()
    with z.AdamW([n], hp, z.AdamWOptions(state_bits=8, seed=5)) as opt:
        opt.step([grad], [param], master, m, v, scales)
        torch.cuda.synchronize()
    tail = entries - first
    g = torch.zeros(tail, device="cuda")
    g[:n - first] = grad[first:].float()
    zero = torch.zeros(tail, device="cuda")
    w, wm, wv = ap.step(g, zero, zero, zero, hp, 1, torch.ones(tail, dtype=torch.bool, device="cuda"), None)
    place = torch.arange(first, entries, device="cuda")
    key = ap.mix(ap.mix(ap.mix(5) ^ 0) ^ 1)
    high = ap.mix((key + 1) & 0xFFFFFFFF)
    h = ap.mix((place & 0xFFFFFFFF) ^ torch.where(place >> 32 > 0, high, key))
    km, sm = ap.encode(wm, ap.M_TOP, 3, h & 0xFFFF, False)
    kr, sr = ap.encode(wv.sqrt(), ap.R_TOP, 4, h >> 16, True)
    live = slice(0, n - first)
    assert torch.equal(master[first:n], w[live]) and torch.equal(param[first:], w[live].bfloat16())
    assert torch.equal(m[first:n].long(), torch.where(wm < 0, km + 128, km)[live])
    assert torch.equal(v[first:n].long(), kr[live])
    assert torch.equal(scales.view(-1, 2)[first // 256:], torch.stack([sm, sr], 1))
    assert not bool(master[:1 << 20].any()) and not bool(m[1 << 31:(1 << 31) + (1 << 20)].any())


def test_two_handles_on_two_streams():
    cases = [Case([70000, 33], bits=bits, seed=9) for bits in (8, 32)]
    twins = [Case([70000, 33], bits=bits, seed=9) for bits in (8, 32)]
    streams = [torch.cuda.Stream() for _ in cases]
    for c, t in zip(cases, twins):
        c.draw()
        t.draw()
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.run(s)
        for t in twins:
            t.run()
    torch.cuda.synchronize()
    for c, t in zip(cases, twins):
        assert torch.equal(c.master, t.master) and torch.equal(c.m, t.m) and torch.equal(c.v, t.v)


def test_refusals():
    c = Case([300, 40], bits=8)
    c.draw()
    args = lambda **k: {**dict(grad_ptrs=c.grads, param_ptrs=c.params, master=c.master, m=c.m, v=c.v, scales=c.scales), **k}  # noqa: E731
    h = c.opt.handle
    for bad, word in ((args(param_ptrs=[c.params[0], c.params[0][10:50]]), "shares memory"),
                      (args(grad_ptrs=[c.params[0], c.grads[1]]), "shares memory"),
                      (args(grad_ptrs=c.grads[:1]), "pointers given"),
                      (args(grad_ptrs=[c.grads[0][:299], c.grads[1]]), "elements"),
                      (args(grad_ptrs=[c.grads[0].float(), c.grads[1]]), "expected torch.bfloat16"),
                      (args(param_ptrs=[c.params[0].cpu(), c.params[1]]), "CUDA"),
                      (args(param_ptrs=[None, c.params[1]]), "NULL"),
                      (args(master=None), "master"), (args(scales=None), "scales"), (args(m=None), "NULL"),
                      (args(m=c.m.float()), "uint8"), (args(scales=c.scales[:-1]), "elements"),
                      (args(v=c.m), "share memory"), (args(scales=c.master[:c.scales.numel()]), "share memory"),
                      (args(master=c.master.data_ptr() + 4), "aligned"),
                      (args(grad_ptrs=[c.grads[0].data_ptr() + 1, c.grads[1]]), "aligned")):
        with pytest.raises(z.Zero1Error, match=word):
            z.zero1_adamw_step(h, **bad)
    # in any order of addresses, and gradients between parameters
    pool = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    for p0, p1, g0, g1, fine in ((0, 512, 1024, 2048, True), (512, 0, 2048, 1024, True), (0, 1024, 512, 2048, True),
                                 (1024, 2048, 0, 512, True), (0, 292, 1024, 2048, False), (292, 260, 1024, 2048, False),
                                 (0, 512, 292, 2048, False), (0, 512, 2048, 544, False), (1000, 0, 700, 36, False)):
        call = dict(param_ptrs=[pool[p0:p0 + 300], pool[p1:p1 + 40]], grad_ptrs=[pool[g0:g0 + 300], pool[g1:g1 + 40]])
        if fine:
            z.zero1_adamw_step(h, **args(**call))
        else:
            with pytest.raises(z.Zero1Error, match="shares memory"):
                z.zero1_adamw_step(h, **args(**call))
    c = Case([300, 40], bits=8)    # one that has not stepped
    c.draw()
    args = lambda **k: {**dict(grad_ptrs=c.grads, param_ptrs=c.params, master=c.master, m=c.m, v=c.v, scales=c.scales), **k}  # noqa: E731
    # a table of pointers is refused the same way
    with pytest.raises(z.Zero1Error, match="elements"):
        c.opt.step(z.PtrTable([c.grads[0][:299], c.grads[1]]), c.params, c.master, c.m, c.v, c.scales)
    with pytest.raises(z.Zero1Error, match="elements"):
        c.opt.moments(c.m, c.v, c.scales, torch.empty(10, device="cuda"))
    big = torch.zeros(2 * c.n, device="cuda")
    for outs in ((big[:c.n], big[256:]), (c.scales.data_ptr(), None)):
        with pytest.raises(z.Zero1Error, match="share"):
            c.opt.moments(c.m, c.v, c.scales, *outs)
    with pytest.raises(z.Zero1Error, match="lr"):
        c.opt.set_lr(-1.0)
    f = Case([10], "f32", "f32", hp=z.Hparams(max_norm=0.0))
    with pytest.raises(z.Zero1Error, match="forms no norm"):
        f.opt.grad_norm()
    with pytest.raises(z.Zero1Error, match="fp32 already"):
        z.zero1_adamw_moments(f.opt.handle, f.m, f.v, torch.zeros(4, device="cuda"), None, None)
    with pytest.raises(z.Zero1Error, match="master"):
        z.zero1_adamw_step(f.opt.handle, f.grads, f.params, torch.zeros(256, device="cuda"), f.m, f.v)
    # nothing ran: the step count is what it was
    assert c.opt.steps() == 0 and f.opt.steps() == 0
    want = c.plain()
    c.run()
    c.check(want)
    h = c.opt.handle
    c.opt.close()
    with pytest.raises(z.Zero1Error, match="invalid handle"):
        z.zero1_adamw_step(h, **args())
