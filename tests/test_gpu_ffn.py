"""The gated feed-forward block on the GPU against 64 bits, within bounds that
tests/ffn_plain.py derives from the roundings, and by norm."""
import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import ffn_plain as fp

pytestmark = pytest.mark.gpu

ACT = {"silu": z.ACT_SILU, "gelu": z.ACT_GELU, "gelu_tanh": z.ACT_GELU_TANH, "relu": z.ACT_RELU}
BF = torch.bfloat16
# By norm: a result rounded once is off by at most 2^-8 / sqrt(3) (errors spread evenly over half a step of entries at
# a power of two; less elsewhere); one whose terms were rounded too, independently, by sqrt(2) times that, and both
# parts of a sum by no more.  2^-8 / sqrt(3) * sqrt(2) = 3.2e-3.
NORM = 3.3e-3


class Matrix:
    """rows x cols of bf16 with `pad` entries between rows, `off` entries past a
    16-byte boundary, between guards that must stay."""

    def __init__(self, rows, cols, pad, off, gen, scale):
        self.shape, self.ld, self.off = (rows, cols), cols + pad, off
        self.full = torch.full((64 + off + rows * self.ld + 64,), 7.0, dtype=BF, device="cuda")
        self.t = torch.as_strided(self.full, self.shape, (self.ld, 1), 64 + off)
        if scale is not None:
            self.t.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * scale)
        else:
            self.t.fill_(float("nan"))     # an output: every entry must be written
        self.mask = torch.ones_like(self.full, dtype=torch.bool)
        torch.as_strided(self.mask, self.shape, (self.ld, 1), 64 + off).fill_(False)

    def intact(self):
        return bool((self.full[self.mask] == 7.0).all())


class Block:
    def __init__(self, rows, width, hidden, name="silu", pad=0, off=0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.name = name
        mk = lambda r, c, s=None: Matrix(r, c, pad, off, gen, s)  # noqa: E731
        self.x, self.dy = mk(rows, width, 1.0), mk(rows, width, 1.0)
        self.w_gate, self.w_up = mk(width, hidden, width ** -0.5), mk(width, hidden, width ** -0.5)
        self.w_down = mk(hidden, width, hidden ** -0.5)
        self.gate, self.up, self.h, self.y = mk(rows, hidden), mk(rows, hidden), mk(rows, hidden), mk(rows, width)
        self.dx, self.dw_gate, self.dw_up = mk(rows, width), mk(width, hidden), mk(width, hidden)
        self.dw_down = mk(hidden, width)
        self.shape = z.FfnShape(rows, width, hidden, ACT[name], width + pad, width + pad, hidden + pad, hidden + pad,
                                hidden + pad, width + pad, unaligned=off % 8 != 0)
        self.errors = torch.zeros(1, dtype=torch.int32, device="cuda")

    def space(self, backward):
        # of the exact size, between guards
        n = z.zero1_ffn_workspace(self.shape, backward)
        full = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        self.guard = (full, n)
        return full[512:512 + n]

    def space_intact(self):
        full, n = self.guard
        return bool((full[:512] == 0xA5).all()) and bool((full[512 + n:] == 0xA5).all())

    def forward(self, train=True, stream=None, space=None):
        z.zero1_ffn_forward(self.shape, self.x.t, self.w_gate.t, self.w_up.t, self.w_down.t,
                            self.gate.t if train else None, self.up.t if train else None, self.h.t, self.y.t,
                            self.space(False) if space is None else space, stream, self.errors)

    def backward(self, dx=True, stream=None, space=None):
        z.zero1_ffn_backward(self.shape, self.dy.t, self.x.t, self.w_gate.t, self.w_up.t, self.w_down.t, self.gate.t,
                             self.up.t, self.h.t, self.dx.t if dx else None, self.dw_gate.t, self.dw_up.t, self.dw_down.t,
                             self.space(True) if space is None else space, stream, self.errors)

    def check(self, want, names):
        for n in names:
            got, (value, off) = getattr(self, n), want[n]
            diff = (got.t.double() - value).abs()
            bad = ~(diff <= off)
            assert not bool(bad.any()), (n, int(bad.sum()), bad.nonzero()[0].tolist(), float(diff.nan_to_num(9e9).max()))
            norm = float(value.norm())
            assert value.numel() < 64 or float(diff.norm()) <= NORM * norm, (n, float(diff.norm()) / norm)
        assert int(self.errors) == 0
        for n, m in vars(self).items():
            if isinstance(m, Matrix):
                assert m.intact(), n
        assert self.space_intact()

    def check_forward(self, train=True):
        want = fp.forward(self.x.t, self.w_gate.t, self.w_up.t, self.w_down.t, self.name)
        self.check(want, ("gate", "up", "h", "y") if train else ("h", "y"))
        if not train:
            assert bool(self.gate.t.isnan().all()) and bool(self.up.t.isnan().all())

    def check_backward(self, dx=True):
        want = fp.backward(self.dy.t, self.x.t, self.w_gate.t, self.w_up.t, self.w_down.t, self.gate.t, self.up.t,
                           self.h.t, self.name)
        self.check(want, (("dx",) if dx else ()) + ("dw_gate", "dw_up", "dw_down"))


SIZES = [
    (1, 8, 8, 0, 0), (1, 1, 1, 0, 1), (1, 768, 2048, 0, 0), (2, 3, 5, 0, 0), (3, 64, 64, 0, 0), (4, 1000, 333, 8, 0),
    (5, 72, 520, 0, 0), (8, 513, 129, 0, 3), (9, 256, 688, 0, 0), (16, 2048, 256, 8, 0), (17, 136, 200, 0, 0),
    (63, 64, 128, 0, 0), (64, 65, 127, 0, 0), (127, 100, 130, 8, 0), (128, 256, 128, 0, 0), (129, 300, 257, 1, 0),
    (255, 256, 256, 0, 0), (257, 517, 1365, 2, 0), (300, 40, 2000, 0, 5), (513, 768, 96, 8, 0), (1003, 264, 136, 0, 0),
]


@pytest.mark.parametrize("name", fp.ACTS)
@pytest.mark.parametrize("rows,width,hidden,pad,off", SIZES)
def test_forward(rows, width, hidden, pad, off, name):
    b = Block(rows, width, hidden, name, pad, off)
    b.forward()
    b.check_forward()
    c = Block(rows, width, hidden, name, pad, off)
    c.forward(train=False)
    c.check_forward(train=False)
    assert torch.equal(b.y.t, c.y.t)


@pytest.mark.parametrize("name", fp.ACTS)
@pytest.mark.parametrize("rows,width,hidden,pad,off", SIZES)
def test_backward(rows, width, hidden, pad, off, name):
    b = Block(rows, width, hidden, name, pad, off)
    b.forward()
    b.backward()
    b.check_backward()


@pytest.mark.parametrize("rows,width,hidden", [(2048, 1024, 2816), (5000, 520, 1032), (700, 2048, 5504)])
def test_many_tiles(rows, width, hidden):
    b = Block(rows, width, hidden)
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()
    first = [m.t.clone() for m in (b.y, b.dx, b.dw_gate, b.dw_up, b.dw_down)]
    b.forward()
    b.backward()
    for a, m in zip(first, (b.y, b.dx, b.dw_gate, b.dw_up, b.dw_down)):
        assert torch.equal(a, m.t)


def test_long_sums():
    """150,000 rows: more than one slice's 65,536, whatever the tiles."""
    b = Block(150000, 136, 264)
    b.forward()
    b.backward()
    b.check_backward()


@pytest.mark.parametrize("rows", [5, 130])
def test_wide_hidden_sums(rows):
    """A hidden size past 65,536: y and dx in slices."""
    b = Block(rows, 24, 70000)
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()


@pytest.mark.parametrize("rows,width,hidden", [(7, 65536, 40), (40, 65000, 16), (130, 65536, 8), (7, 24, 65536)])
def test_widest(rows, width, hidden):
    b = Block(rows, width, hidden)
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()


def test_backward_without_dx():
    b = Block(200, 96, 160)
    b.forward()
    b.backward(dx=False)
    b.check_backward(dx=False)
    assert bool(b.dx.t.isnan().all())


def test_no_rows():
    b = Block(0, 40, 24, pad=8)
    b.forward()
    b.backward()
    for m in (b.dw_gate, b.dw_up, b.dw_down):
        assert bool((m.t == 0).all()) and m.intact()


def test_column_slices():
    """Wg and Wu (and their gradients) as halves of one matrix, gate, up and h
    as thirds of one buffer."""
    rows, width, hidden = 300, 128, 160
    b = Block(rows, width, hidden)
    w = torch.cat([b.w_gate.t, b.w_up.t], 1).contiguous()
    dw = torch.full_like(w, math.nan)
    acts = torch.full((rows, 3 * hidden), math.nan, dtype=BF, device="cuda")
    s = z.FfnShape(rows, width, hidden, ldh=3 * hidden, ld_gate=2 * hidden, ld_up=2 * hidden)
    gate, up, h = acts[:, :hidden], acts[:, hidden:2 * hidden], acts[:, 2 * hidden:]
    space = torch.empty(z.zero1_ffn_workspace(s, True), dtype=torch.uint8, device="cuda")
    z.zero1_ffn_forward(s, b.x.t, w[:, :hidden], w[:, hidden:], b.w_down.t, gate, up, h, b.y.t, space)
    z.zero1_ffn_backward(s, b.dy.t, b.x.t, w[:, :hidden], w[:, hidden:], b.w_down.t, gate, up, h, b.dx.t, dw[:, :hidden],
                         dw[:, hidden:], b.dw_down.t, space)
    c = Block(rows, width, hidden)
    c.forward()
    c.backward()
    for x, y in ((gate, c.gate.t), (up, c.up.t), (h, c.h.t), (b.y.t, c.y.t), (b.dx.t, c.dx.t), (dw[:, :hidden], c.dw_gate.t),
                 (dw[:, hidden:], c.dw_up.t), (b.dw_down.t, c.dw_down.t)):
        assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """gate, up and h with rows 2^24 entries apart: 300 rows reach past 2^32 entries."""
    rows, width, hidden, ld = 300, 64, 72, 1 << 24
    b = Block(rows, width, hidden)
    s = z.FfnShape(rows, width, hidden, ldh=ld)
    big = torch.empty(rows * ld, dtype=BF, device="cuda")
    gate, up, h = (torch.as_strided(big, (rows, hidden), (ld, 1), 128 * i) for i in range(3))
    space = torch.empty(z.zero1_ffn_workspace(s, True), dtype=torch.uint8, device="cuda")
    z.zero1_ffn_forward(s, b.x.t, b.w_gate.t, b.w_up.t, b.w_down.t, gate, up, h, b.y.t, space)
    z.zero1_ffn_backward(s, b.dy.t, b.x.t, b.w_gate.t, b.w_up.t, b.w_down.t, gate, up, h, b.dx.t, b.dw_gate.t, b.dw_up.t,
                         b.dw_down.t, space)
    c = Block(rows, width, hidden)
    c.forward()
    c.backward()
    for x, y in ((gate, c.gate.t), (h, c.h.t), (b.y.t, c.y.t), (b.dx.t, c.dx.t), (b.dw_down.t, c.dw_down.t)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_row_that_is_not_finite_stays_alone(rows, bad):
    b = Block(rows, 96, 136)
    b.x.t[1, 5] = bad
    b.forward()
    fine = [i for i in range(rows) if i != 1]
    c = Block(rows, 96, 136)
    c.forward()
    for m, n in ((b.y, c.y), (b.h, c.h), (b.gate, c.gate)):
        assert torch.equal(m.t[fine], n.t[fine])
    assert not bool(b.y.t[1].isfinite().any())


def test_large_gates_stay_finite():
    """Gates of plus and minus 200: the exponential overflows, the block does not."""
    for name in fp.ACTS:
        b = Block(200, 64, 72, name)
        b.w_gate.t.mul_(60)
        b.forward()
        b.check_forward()
        b.backward()
        b.check_backward()


@pytest.mark.parametrize("rows", [1, 400])
def test_captured_calls_on_another_stream(rows):
    a, b = Block(rows, 264, 520, "gelu", 1), Block(rows, 264, 520, "gelu", 1)
    a.forward()
    a.backward()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    spaces = [b.space(k) for k in (False, True)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cur = torch.cuda.current_stream()
        b.forward(stream=cur, space=spaces[0])
        b.backward(stream=cur, space=spaces[1])
    keep = b.x.t.clone()
    b.x.t.zero_()
    with torch.cuda.stream(s):
        graph.replay()
        b.x.t.copy_(keep)
        graph.replay()
    s.synchronize()
    for n in ("y", "h", "dx", "dw_gate", "dw_up", "dw_down"):
        assert torch.equal(getattr(a, n).t, getattr(b, n).t), n


def test_two_streams_at_once():
    """Calls whose workspaces are their own may overlap."""
    blocks = [Block(600, 256, 512, seed=i) for i in range(2)]
    twins = [Block(600, 256, 512, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in blocks]
    spaces = [[b.space(k) for k in (False, True)] for b in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, sp in zip(blocks, streams, spaces):
            b.forward(stream=s, space=sp[0])
            b.backward(stream=s, space=sp[1])
    torch.cuda.synchronize()
    for b, t in zip(blocks, twins):
        t.forward()
        t.backward()
        for n in ("y", "dx", "dw_gate", "dw_up", "dw_down"):
            assert torch.equal(getattr(b, n).t, getattr(t, n).t), n


def test_gradient_against_differences():
    """<gradient, direction> against central differences of <dy, y> in 64 bits
    at the bf16 inputs: the gradient's own roundings are at most 2^-8 by norm
    (NORM) of the gradient; the directions are random, so each inner product
    is off by some NORM |gradient| |direction| / sqrt(entries), here bounded by
    6 of those."""
    rows, width, hidden = 200, 64, 96
    b = Block(rows, width, hidden, "silu")
    b.forward()
    b.backward()
    t = {n: getattr(b, n).t.double() for n in ("x", "w_gate", "w_up", "w_down", "dy")}

    def loss(v):
        return float((fp.act(v["x"] @ v["w_gate"], "silu")[0] * (v["x"] @ v["w_up"]) @ v["w_down"] * t["dy"]).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for key, out in (("x", "dx"), ("w_gate", "dw_gate"), ("w_up", "dw_up"), ("w_down", "dw_down")):
        d = torch.randn(t[key].shape, generator=gen, device="cuda", dtype=torch.float64)
        eps = 1e-5
        diff = (loss({**t, key: t[key] + eps * d}) - loss({**t, key: t[key] - eps * d})) / (2 * eps)
        g = getattr(b, out).t.double()
        # the saved gate, up and h are rounded too: as much again
        assert abs(diff - float((g * d).sum())) <= 6 * 2 * NORM * float(g.norm()), key


@pytest.mark.parametrize("rows", [5, 300])
def test_a_wait_that_runs_out_is_reported(rows):
    b = Block(rows, 64, 64)
    s = z.FfnShape(rows, 64, 64, inject_wait_timeout=True)
    z.zero1_ffn_forward(s, b.x.t, b.w_gate.t, b.w_up.t, b.w_down.t, b.gate.t, b.up.t, b.h.t, b.y.t, b.space(False), None,
                        b.errors)
    assert int(b.errors) == 1
    b.errors.zero_()
    b.forward()
    b.check_forward()


def test_refusals():
    b = Block(40, 64, 72)
    args = dict(shape=b.shape, x=b.x.t, w_gate=b.w_gate.t, w_up=b.w_up.t, w_down=b.w_down.t, gate=b.gate.t, up=b.up.t,
                h=b.h.t, y=b.y.t, workspace=b.space(False))
    for kw, word in ((dict(x=b.x.t.float()), "expected torch.bfloat16"), (dict(x=b.x.t.cpu()), "CUDA"),
                     (dict(y=b.y.t[:39]), "expected 40 x 64"), (dict(w_down=b.w_down.t[:, :-1]), "expected 72 x 64"),
                     (dict(x=b.x.t.t()), "expected 40 x 64"), (dict(y=torch.empty(40 * 64 - 1, dtype=BF, device="cuda")), "elements"),
                     (dict(x=torch.empty(40, 128, dtype=BF, device="cuda")[:, ::2]), "adjacent"),
                     (dict(h=torch.empty(40, 80, dtype=BF, device="cuda")[:, :72]), "stride"), (dict(workspace=torch.empty(8)), "CUDA"),
                     (dict(y=b.x.t), "share"), (dict(up=None), "together")):
        with pytest.raises(z.Zero1Error, match=word):
            z.zero1_ffn_forward(**{**args, **kw})
    assert bool(b.y.t.isnan().all())
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(z.Zero1Error, match="lies in the workspace"):
        z.zero1_ffn_forward(**{**args, "y": space[4096:4096 + 40 * 64 * 2].view(BF).view(40, 64), "workspace": space})
    odd = Block(40, 65, 72)
    with pytest.raises(z.Zero1Error, match="workspace holds"):
        z.zero1_ffn_forward(odd.shape, odd.x.t, odd.w_gate.t, odd.w_up.t, odd.w_down.t, None, None, odd.h.t, odd.y.t,
                            torch.empty(100, dtype=torch.uint8, device="cuda"))
