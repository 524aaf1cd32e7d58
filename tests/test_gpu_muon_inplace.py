"""One buffer as input and output of the orthogonalisation: taken with one
type, refused with two (entries lie at other places then, and a block could
write where another has yet to read)."""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mats", [[(0, 64, 64), (4096, 64, 64)], [(0, 200, 300)]])
def test_two_types_in_one_buffer_are_refused(mats):
    n = 200 * 300
    x = torch.randn(n, device="cuda")
    before = x.clone()
    low = x.view(torch.bfloat16)
    with z.Muon(n, 1, mats) as opt:
        for src, a, dst, b in ((low, z.DTYPE_BF16, x, z.DTYPE_F32), (x, z.DTYPE_F32, low, z.DTYPE_BF16)):
            with pytest.raises(z.Zero1Error) as e:
                z.zero1_muon_orthogonalize(opt.handle, src, a, dst, b)
            assert e.value.code == -1 and "types" in str(e.value)
        torch.cuda.synchronize()
        assert torch.equal(x, before)
        want = torch.empty_like(x)
        opt.orthogonalize(x, want)
        opt.orthogonalize(x, x)
        opt.status()
        for off, r, c in mats:
            assert torch.equal(x[off:off + r * c], want[off:off + r * c])
