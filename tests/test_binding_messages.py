"""What the binding says of a wrong buffer: which argument, and which of the
W ranks' buffers it is."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import zero_sharded_adamw_gb300 as z


class Device:
    """A CPU tensor that says it is on the device; only checks look at it."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def good():
    return Device(torch.zeros(16, dtype=torch.bfloat16))


@pytest.mark.parametrize("bad", [torch.zeros(16, dtype=torch.bfloat16), Device(torch.zeros(16)),
                                 Device(torch.zeros(15, dtype=torch.bfloat16)),
                                 Device(torch.zeros(32, dtype=torch.bfloat16)[::2]), np.zeros(16, np.uint16)])
@pytest.mark.parametrize("rank", [0, 2])
@pytest.mark.parametrize("table", [False, True])
def test_the_rank_of_a_wrong_buffer_is_named(bad, rank, table):
    xs = [good() for _ in range(3)]
    xs[rank] = bad
    if table:
        if isinstance(bad, np.ndarray):
            pytest.skip("a pointer table of a host array")
        xs = z.PtrTable(xs)
    with pytest.raises(z.Zero1ArgumentError) as e:
        z._ptrs(xs, 3, 16, "bf16", True, "grads")
    assert str(e.value).startswith(f"ZERO1_EINVAL: grads[{rank}]: "), e.value


def test_through_an_entry_point():
    cpu = [torch.zeros(8, dtype=torch.float32) for _ in range(2)]
    with pytest.raises(z.Zero1ArgumentError, match=r": in\[0\]: "):
        z.zero1_allreduce(8, 2, z.DTYPE_F32, 0, cpu, cpu)


def test_good_buffers_pass():
    xs = [good() for _ in range(3)]
    assert list(z._ptrs(xs, 3, 16, "bf16", True, "grads")) == [x.data_ptr() for x in xs]
