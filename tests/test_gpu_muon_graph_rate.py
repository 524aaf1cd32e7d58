"""The learning rate of a captured matrix step is the one it was captured
with; a later rate reaches later calls only."""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(64, 64), (200, 300)])
def test_a_captured_step_keeps_its_rate(shape):
    n = shape[0] * shape[1]
    g = torch.Generator(device="cuda").manual_seed(n)
    grads = [torch.randn(n, generator=g, device="cuda").to(torch.bfloat16)]
    params = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    start = 0.02 * torch.randn(n, generator=g, device="cuda")

    def moved(lr, call):
        master.copy_(start)
        momentum.zero_()
        opt.set_lr(lr)
        call()
        opt.status()
        return master.clone()

    master, momentum = start.clone(), torch.zeros(n, device="cuda")
    with z.Muon(n, 1, [(0, *shape)], z.MuonHparams(lr=1e-2)) as opt:
        def step():
            opt.step(grads, params, master, momentum, torch.cuda.current_stream())
        slow, fast = moved(1e-3, step), moved(1e-2, step)
        graph = torch.cuda.CUDAGraph()
        opt.set_lr(1e-2)
        with torch.cuda.graph(graph):
            step()
        assert not torch.equal(slow, fast)
        assert torch.equal(moved(1e-3, graph.replay), fast)
        assert torch.equal(moved(1e-3, step), slow)
