"""The binding's check of a row stride against the tensor it is given for."""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z


class Device:
    """A CPU tensor that says it is on the device; only its shape is looked at."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("make,ld", [
    (lambda b: b[:4, :8], 8),               # padded rows taken for dense ones
    (lambda b: b[::2, :8][:4], 12),         # every other row taken for each
    (lambda b: b.view(-1)[:32].view(4, 8), 12)])
def test_rows_of_another_stride_are_refused(make, ld):
    x = make(torch.zeros(16, 12))
    assert x.shape == (4, 8) and x.stride(0) != ld
    with pytest.raises(z.Zero1ArgumentError, match="row stride"):
        z._take_rows(Device(x), 4, 8, ld, "f32", "x")
    assert z._take_rows(Device(x), 4, 8, x.stride(0), "f32", "x") == x.data_ptr()


def test_other_shapes_say_nothing_of_the_stride():
    base = torch.zeros(16, 12)
    for x, rows, ld in ((base, 8, 24), (base.view(-1), 4, 12), (base.view(4, 4, 12), 16, 12), (base[:1, :8], 1, 8),
                        (base, 5, 12)):
        assert z._take_rows(Device(x), rows, 8, ld, "f32", "x") == x.data_ptr()
    one = base[:1, :8]                      # a single row has no stride to keep
    assert one.shape == (1, 8) and one.stride(0) == 12
