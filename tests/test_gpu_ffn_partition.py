"""The feed-forward block on the streams of an SM partition, whose SMs may not
hold the clusters that the whole device does."""
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_gpu_ffn import Block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [8, 120])
@pytest.mark.parametrize("rows", [1, 20, 100, 300])
def test_forward_and_backward_on_either_part(sms, rows):
    with z.SmPartition(sms) as part:
        for raw in (part.stream_a, part.stream_b):
            s = torch.cuda.ExternalStream(raw)
            b = Block(rows, 520, 1032)
            spaces = [b.space(k) for k in (False, True)]
            torch.cuda.synchronize()
            b.forward(stream=s, space=spaces[0])
            b.backward(stream=s, space=spaces[1])
            s.synchronize()
            b.check_forward()
            b.check_backward()
