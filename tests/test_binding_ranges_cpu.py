"""Numbers that do not fit the C fields of the feed-forward block's and the
list step's calls are refused, not cut off."""
import pytest

import zero_sharded_adamw_gb300 as z


@pytest.mark.parametrize("bad", [1 << 32, (1 << 32) + z.ACT_GELU, -(1 << 32), 1 << 31, 1 << 64])
def test_activation(bad):
    with pytest.raises(z.Zero1ArgumentError, match="activation"):
        z.zero1_ffn_workspace(z.FfnShape(4, 16, 32, bad))


@pytest.mark.parametrize("field,bad", [("state_bits", (1 << 32) + 8), ("state_bits", (1 << 32) + 32), ("state_bits", 8 - (1 << 32)),
                                       ("param_dtype", 1 << 32), ("grad_dtype", (1 << 32) + 1), ("grad_dtype", 1 << 64)])
def test_adamw_options(field, bad):
    opts = z.AdamWOptions()
    setattr(opts, field, bad)
    with pytest.raises(z.Zero1ArgumentError, match=field):
        z.zero1_adamw_create((4,), None, opts)


@pytest.mark.parametrize("bad", [-1, 1 << 64, -(1 << 64) + 3])
def test_steps(bad):
    with pytest.raises(z.Zero1ArgumentError, match="steps"):
        z.zero1_adamw_set_steps(12345, bad)


def test_numbers_that_fit_reach_the_library():
    for bad in (4, -1, (1 << 31) - 1, -(1 << 31)):
        with pytest.raises(z.Zero1Error, match="unknown activation"):
            z.zero1_ffn_workspace(z.FfnShape(4, 16, 32, bad))
    with pytest.raises(z.Zero1Error, match="state_bits must be"):
        z.zero1_adamw_create((4,), None, z.AdamWOptions(state_bits=-1))
    for t in (0, (1 << 64) - 1):
        with pytest.raises(z.Zero1Error, match="invalid handle"):
            z.zero1_adamw_set_steps(12345, t)
