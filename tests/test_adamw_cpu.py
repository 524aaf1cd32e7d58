"""AdamW over many tensors: what is refused, and the 8-bit codes' formulas,
without a GPU."""
import ctypes as C

import numpy as np
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import adamw_plain as ap


def create(sizes=(4,), hp=None, opts=None, decays=None):
    return z.zero1_adamw_create(sizes, hp or z.Hparams(), opts or z.AdamWOptions(), decays)


@pytest.mark.parametrize("kw,word", [
    (dict(sizes=()), "count"),
    (dict(sizes=(0, 0)), "empty"),
    (dict(sizes=(1 << 41,)), "2\\^40"),
    (dict(sizes=(1 << 40, 1 << 40)), "2\\^40"),
    (dict(opts=z.AdamWOptions(state_bits=16)), "state_bits"),
    (dict(opts=z.AdamWOptions(param_dtype=2)), "dtype"),
    (dict(opts=z.AdamWOptions(grad_dtype=-1)), "dtype"),
    (dict(hp=z.Hparams(lr=-1.0)), "lr"),
    (dict(hp=z.Hparams(lr=float("nan"))), "lr"),
    (dict(hp=z.Hparams(beta1=1.0)), "betas"),
    (dict(hp=z.Hparams(beta2=-0.1)), "betas"),
    (dict(hp=z.Hparams(eps=float("inf"))), "eps"),
    (dict(hp=z.Hparams(weight_decay=-0.1)), "weight_decay"),
    (dict(hp=z.Hparams(max_norm=float("nan"))), "max_norm"),
    (dict(hp=z.Hparams(beta2=0.999999)), "bias corrections"),
])
def test_create_refuses(kw, word):
    with pytest.raises(z.Zero1Error, match=word) as e:
        create(**kw)
    assert e.value.code == -1


def test_binding_refuses():
    with pytest.raises(z.Zero1ArgumentError, match="decays"):
        create((3, 4), decays=[True])
    with pytest.raises(z.Zero1ArgumentError, match="sizes"):
        create((-1,))
    with pytest.raises(z.Zero1ArgumentError, match="seed"):
        create(opts=z.AdamWOptions(seed=-1))


def test_c_entry_refuses_before_any_device_call():
    lib = z._load()
    sizes, out = (C.c_uint64 * 1)(4), C.c_void_p(7)
    hp, o = z.Hparams()._c(), z.AdamWOptions()._c()
    assert lib.zero1_adamw_create(sizes, None, 1, C.byref(hp), C.byref(o), None) == -1
    assert lib.zero1_adamw_create(None, None, 1, C.byref(hp), C.byref(o), C.byref(out)) == -1 and out.value is None
    assert lib.zero1_adamw_create(sizes, None, 1, None, C.byref(o), C.byref(out)) == -1
    assert lib.zero1_adamw_create(sizes, None, 65537, C.byref(hp), C.byref(o), C.byref(out)) == -1
    for field, v in (("size", 8), ("reserved", 1), ("decay_before_update", 2)):
        bad = z.AdamWOptions()._c()
        setattr(bad, field, v)
        assert lib.zero1_adamw_create(sizes, None, 1, C.byref(hp), C.byref(bad), C.byref(out)) == -1, field
    assert lib.zero1_adamw_destroy(None) == 0
    for f, args in (("destroy", ()), ("step", (None,) * 7), ("moments", (None,) * 6), ("set_steps", (1, None)),
                    ("set_lr", (0.1, None)), ("get_steps", (None, None)), ("get_grad_norm", (None, None, None)),
                    ("layout", (None, None, None))):
        assert getattr(lib, "zero1_adamw_" + f)(C.c_void_p(12345), *args) == -1, f


def test_codes_are_increasing_and_reach_the_top():
    for bits, top in ((3, ap.M_TOP), (4, ap.R_TOP)):
        f = ap.value(torch.arange(16 * 2 ** bits), bits)
        assert f[0] == 0 and f[-1] == top and bool((f[1:] > f[:-1]).all())
        # steps are a fraction 2^-(bits+1) .. 2^-bits of value + 1
        gap = (f[1:] - f[:-1]) / (f[:-1] + 1)
        assert gap.max() <= 2.0 ** -bits and gap.min() > 2.0 ** -(bits + 1)


@pytest.mark.parametrize("bits,top", [(3, ap.M_TOP), (4, ap.R_TOP)])
def test_random_rounding_is_between_its_neighbours_and_unbiased(bits, top):
    """Over the 65,536 dithers an entry can get, the mean of what its code
    stands for is the entry: to 2^-16 of the code's width (the dither is a
    multiple of 2^-16 of it) and the rounding of x inv + 1 and of the scale
    (2^-24 each of value + 1, in block units)."""
    g = torch.Generator().manual_seed(0)
    x = torch.exp(-6 * torch.rand(BLOCK := ap.BLOCK, generator=g))
    x[0], x[1], x[2] = 1.0, 0.0, 2.0 ** -19
    every = torch.arange(0, 65536, 16)
    total = torch.zeros(BLOCK, dtype=torch.float64)
    for d in every:
        k, scale = ap.encode(x, top, bits, torch.full((BLOCK,), int(d)), False)
        q = ap.value(k, bits) * scale.double()
        total += q
        width = (ap.value(k, bits) - ap.value((k - 1).clamp(min=0), bits)) * scale.double()   # to the code below
        slack = (q + scale.double()) * 2.0 ** -21
        assert bool((q <= x.double() + torch.maximum(width, slack) + slack).all())
    mean = total / len(every)
    width = (x.double() + float(scale)) * 2.0 ** -bits
    # 4,096 of the dithers: the mean is off by up to 2^-12 of the width
    assert bool(((mean - x.double()).abs() <= width * 2.0 ** -12 + (x.double() + float(scale)) * 2.0 ** -22).all())


def test_plain_hash_is_even():
    """256 bins of 2^20 numbers: their counts' chi-square of 255 degrees stays
    below its mean by 6 standard deviations (22.6)."""
    a, b = ap.dither(1 << 20, 7, 3, "cpu")
    for h in (a, b):
        counts = torch.bincount(h >> 8, minlength=256).double()
        e = (1 << 20) / 256
        assert float(((counts - e) ** 2 / e).sum()) < 255 + 6 * 22.6
    assert abs(float(np.corrcoef(a.numpy(), b.numpy())[0, 1])) < 6 / 1024
