"""The gated feed-forward block without a GPU: refusals, the workspace's size,
and the plain gradients against differences."""
import ctypes as C

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import ffn_plain as fp


@pytest.mark.parametrize("kw,word", [
    (dict(activation=4), "activation"), (dict(activation=-1), "activation"),
    (dict(rows=1 << 31), "rows"), (dict(width=0), "width"), (dict(width=65537), "width"),
    (dict(hidden=0), "hidden"), (dict(hidden=(1 << 20) + 1), "hidden"),
    (dict(ldx=15), "ldx"), (dict(ldy=15), "ldy"), (dict(ldh=31), "ldh"), (dict(ld_gate=31), "ld_gate"),
    (dict(ld_up=31), "ld_up"), (dict(ld_down=15), "ld_down"), (dict(ld_down=1 << 38), "ld_down"),
    (dict(rows=1 << 20, ldx=1 << 31), "ldx"), (dict(rows=(1 << 31) - 1, hidden=1 << 18), "too large"),
])
def test_shapes_refused(kw, word):
    shape = z.FfnShape(**{**dict(rows=4, width=16, hidden=32), **kw})
    with pytest.raises(z.Zero1Error, match=word) as e:
        z.zero1_ffn_workspace(shape)
    assert e.value.code == -1
    for f, count in (("forward", 8), ("backward", 12)):
        assert getattr(z._load(), "zero1_ffn_" + f)(C.byref(shape._c), *([None] * (count + 1)), 0, None, None) == -1


def test_c_entry_refuses():
    lib = z._load()
    shape = z.FfnShape(4, 16, 32)
    b = C.c_uint64()
    assert lib.zero1_ffn_workspace(None, 0, C.byref(b)) == -1
    assert lib.zero1_ffn_workspace(C.byref(shape._c), 0, None) == -1
    for field, v in (("size", 8), ("unaligned", 2), ("inject_wait_timeout", -1)):
        bad = z.FfnShape(4, 16, 32)._c
        setattr(bad, field, v)
        assert lib.zero1_ffn_workspace(C.byref(bad), 0, C.byref(b)) == -1, field
    with pytest.raises(z.Zero1ArgumentError, match="rows"):
        z.FfnShape(-1, 16, 32)


# addresses that nothing dereferences: every refusal comes before a device call
def fake(i, offset=0):
    return (i + 1) * (1 << 24) + offset


def fwd(shape, **kw):
    a = dict(x=fake(0), w_gate=fake(1), w_up=fake(2), w_down=fake(3), gate=fake(4), up=fake(5), h=fake(6), y=fake(7))
    z.zero1_ffn_forward(shape, **{**a, **kw})


def bwd(shape, **kw):
    names = "dy x w_gate w_up w_down gate up h dx dw_gate dw_up dw_down".split()
    z.zero1_ffn_backward(shape, **{**{n: fake(i) for i, n in enumerate(names)}, **kw})


@pytest.mark.parametrize("call,kw,word", [
    (fwd, dict(x=None), "NULL"), (fwd, dict(y=None), "NULL"), (fwd, dict(h=None), "NULL"), (fwd, dict(gate=None), "together"),
    (fwd, dict(x=fake(0, 2)), "x is not 16-byte"), (fwd, dict(y=fake(0)), "x and y share"),
    (fwd, dict(h=fake(1, 16)), "w_gate and h share"), (fwd, dict(up=fake(4)), "gate and up share"),
    (fwd, dict(up=fake(4, 64)), "gate and up share"), (fwd, dict(errors=3), "errors"),
    (bwd, dict(dy=None), "NULL"), (bwd, dict(dw_up=None), "NULL"), (bwd, dict(dx=fake(0)), "dx and dy share"),
    (bwd, dict(dx=fake(1, 32)), "dx and x share"), (bwd, dict(dw_gate=fake(2)), "dw_gate and w_gate share"),
    (bwd, dict(dw_up=fake(9)), "dw_gate and dw_up share"), (bwd, dict(gate=fake(5, 2)), "gate is not"),
])
def test_buffers_refused(call, kw, word):
    with pytest.raises(z.Zero1Error, match=word):
        call(z.FfnShape(40, 16, 32), **kw)


def test_unaligned_buffers_refused_to_the_element():
    with pytest.raises(z.Zero1Error, match="aligned to its elements"):
        fwd(z.FfnShape(40, 16, 32, unaligned=True), x=fake(0, 1))


def test_column_slices_of_one_matrix_share_nothing():
    """Rows equally far apart, side by side: only then the workspace is looked
    at (and refused), not the overlap."""
    shape = z.FfnShape(200, 16, 32, ldh=96, ld_gate=64, ld_up=64)
    slices = dict(w_gate=fake(1), w_up=fake(1, 64), gate=fake(4), up=fake(4, 64), h=fake(4, 128))
    with pytest.raises(z.Zero1Error, match="device query|no CUDA|driver|ECUDA"):
        if torch.cuda.is_available():
            pytest.skip("the call would run")
        fwd(shape, **slices)
    with pytest.raises(z.Zero1Error, match="gate and h share|up and h share|h and gate share|h and up share"):
        fwd(shape, **{**slices, "h": fake(4, 126 - 14)})
    # the last columns of one run into the next row of the other
    with pytest.raises(z.Zero1Error, match="share"):
        fwd(z.FfnShape(200, 16, 32, ldh=96), gate=fake(4), up=fake(4, 160))


def test_workspace():
    dense = z.FfnShape(16384, 4096, 11008)
    assert z.zero1_ffn_workspace(dense) == 0 and z.zero1_ffn_workspace(dense, True) == 2 * 16384 * 11008 * 2
    assert z.zero1_ffn_workspace(z.FfnShape(0, 16, 32), True) == 0
    # odd strides: copies of the operands, rows padded to 8 entries
    odd = z.FfnShape(1000, 517, 1365, ldx=519, ldy=519, ldh=1367, ld_gate=1367, ld_up=1367, ld_down=519)
    base = z.FfnShape(1000, 517, 1365, ldx=520, ldy=520, ldh=1368, ld_gate=1368, ld_up=1368, ld_down=520)
    up = lambda r, c: -(-r * (-(-c // 8) * 8) * 2 // 256) * 256  # noqa: E731
    copies = up(1000, 517) + up(1000, 1365) + 2 * up(517, 1365) + up(1365, 517)
    assert z.zero1_ffn_workspace(odd) - z.zero1_ffn_workspace(base) == copies
    assert z.zero1_ffn_workspace(odd, True) - z.zero1_ffn_workspace(base, True) == copies + up(1000, 517)
    loose = z.FfnShape(**{**{k: getattr(base, k) for k in base.__dataclass_fields__}, "unaligned": True})
    assert z.zero1_ffn_workspace(loose) == z.zero1_ffn_workspace(odd)
    with pytest.raises(z.Zero1Error, match="workspace holds 0 bytes"):
        fwd(odd)


@pytest.mark.parametrize("name", fp.ACTS)
def test_plain_gradients_are_the_differences(name):
    """Central differences of the loss <dy, y> in 64 bits: off by the third
    derivative times step^2 (1e-10) and rounding over the step (1e-11)."""
    g = torch.Generator().manual_seed(3)
    r, w, h = 5, 4, 6
    t = {k: torch.randn(*s, generator=g, dtype=torch.float64)
         for k, s in (("x", (r, w)), ("wg", (w, h)), ("wu", (w, h)), ("wd", (h, w)), ("dy", (r, w)))}

    def loss(v):
        return float((fp.act(v["x"] @ v["wg"], name)[0] * (v["x"] @ v["wu"]) @ v["wd"] * t["dy"]).sum())

    gate, up = t["x"] @ t["wg"], t["x"] @ t["wu"]
    hid = fp.act(gate, name)[0] * up
    grads = fp.backward(t["dy"], t["x"], t["wg"], t["wu"], t["wd"], gate, up, hid, name)
    for key, out in (("x", "dx"), ("wg", "dw_gate"), ("wu", "dw_up"), ("wd", "dw_down")):
        d = torch.randn(t[key].shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        diff = (loss({**t, key: t[key] + eps * d}) - loss({**t, key: t[key] - eps * d})) / (2 * eps)
        assert abs(diff - float((grads[out][0] * d).sum())) <= 1e-7 * (1 + abs(diff)), key
