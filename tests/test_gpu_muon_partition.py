"""The matrix step on the streams of an SM partition.  Matrices stepped by a
cluster of four or eight blocks need that many SMs of one processing cluster:
where a stream has them the results are the whole device's, where it has not
the call is refused before anything is written."""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z

pytestmark = pytest.mark.gpu

# a cluster of one, two, four and eight blocks, and a matrix of tiles
SHAPES = [(64, 64), (100, 300), (64, 700), (900, 40), (128, 1536), (200, 300)]


def total_sms() -> int:
    return torch.cuda.get_device_properties(0).multi_processor_count


def problem():
    mats, at = [], 0
    for r, c in SHAPES:
        mats.append((at, r, c))
        at += (r * c + 7) // 8 * 8
    return mats, torch.randn(at, device="cuda", generator=torch.Generator(device="cuda").manual_seed(12))


@pytest.mark.parametrize("sms_a", [8, 16, 64, 120, 136, 144])
@pytest.mark.parametrize("which", ["stream_a", "stream_b"])
def test_on_a_partition_or_refused(sms_a, which):
    if sms_a >= total_sms():
        pytest.skip("fewer SMs")
    mats, u = problem()
    want = torch.empty_like(u)
    got = torch.full_like(u, 3.0)
    master, momentum = torch.full_like(u, 2.0), torch.full_like(u, 1.0)
    grads, params = [u.to(torch.bfloat16)], [torch.full_like(u, 5.0, dtype=torch.bfloat16)]
    with z.Muon(u.numel(), 1, mats) as opt, z.SmPartition(sms_a) as part:
        opt.orthogonalize(u, want)
        torch.cuda.synchronize()
        stream = getattr(part, which)
        try:
            opt.orthogonalize(u, got, stream)
            opt.status(stream)
            assert torch.equal(got[:mats[-1][0]], want[:mats[-1][0]])
            off, r, c = mats[-1]
            assert torch.equal(got[off:off + r * c], want[off:off + r * c])
        except z.Zero1Error as e:
            # eight blocks of one processing cluster: 8 SMs of the first group always are
            assert which == "stream_b" and e.code == -1 and "cluster of" in str(e)
            with pytest.raises(z.Zero1Error):
                opt.step(grads, params, master, momentum, stream)
            torch.cuda.synchronize()
            assert (got == 3.0).all() and (master == 2.0).all() and (momentum == 1.0).all()
            assert (params[0].float() == 5.0).all()
        opt.orthogonalize(u, got)          # the handle goes on
        opt.status()
        assert all(torch.equal(got[o:o + r * c], want[o:o + r * c]) for o, r, c in mats)


def test_the_smallest_rest_refuses_a_cluster_of_eight():
    """The rest is what the first group left over.  Its 8 SMs lie on several
    processing clusters (then the call is refused) or on one (then it runs),
    by how the driver picked them."""
    with z.SmPartition(total_sms() - 8) as part, z.Muon(64 * 1000, 1, [(0, 64, 1000)]) as opt:
        if part.sms_b > 8:
            pytest.skip("no group of 8 SMs")
        u, out = torch.randn(64 * 1000, device="cuda"), torch.full((64 * 1000,), 3.0, device="cuda")
        try:
            opt.orthogonalize(u, out, part.stream_b)
        except z.Zero1Error as e:
            assert e.code == -1 and "cluster of 8 blocks" in str(e)
            torch.cuda.synchronize()
            assert (out == 3.0).all()
        else:
            opt.status(part.stream_b)
