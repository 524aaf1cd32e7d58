"""Layer norm, the gated feed-forward block and AdamW over a list used together
(examples/train_gated_block.py): the block's gradients against 64 bits and
against differences, and that a run is the same twice."""
import importlib.util
import math
import os

import pytest
import torch

from tests import ffn_plain as fp

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("train_gated_block", os.path.join(ROOT, "examples", "train_gated_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def output64(v, eps):
    """The block in 64 bits."""
    x = v["x"]
    d = x - x.mean(1, keepdim=True)
    n = d / (d.square().mean(1, keepdim=True) + eps).sqrt() * v["gamma"] + v["beta"]
    return x + fp.act(n @ v["w_gate"], "silu")[0] * (n @ v["w_up"]) @ v["w_down"]


@pytest.mark.parametrize("rows,width,hidden", [(300, 64, 96), (64, 136, 200)])
def test_gradients(rows, width, hidden):
    """Gradients by autograd of the 64-bit block at the same bf16 parameters,
    by norm: the chain rounds to bf16 five times at most (n; gate, up and h;
    dgate and dup; dn; the result), each by 2^-8 / sqrt(3) of its norm, and
    differences along a random direction."""
    mod = load()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    block = mod.GatedBlock(width, hidden, rows, gen)
    block.p["gamma"].copy_(1 + 0.2 * torch.randn(width, generator=gen, device="cuda"))
    block.p["beta"].copy_(0.2 * torch.randn(width, generator=gen, device="cuda"))
    x = (torch.randn(rows, width, generator=gen, device="cuda") * 1.5 + 0.3).bfloat16()
    dy = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    y = block.forward(x)
    got = {"x": block.backward(x, dy)} | block.g
    v = {k: t.detach().double().requires_grad_(True) for k, t in ({"x": x} | block.p).items()}
    out = output64(v, mod.EPS)
    (out * dy.double()).sum().backward()
    step = 2.0 ** -8 / math.sqrt(3)
    assert float((y.double() - out.detach()).norm()) <= 4 * step * float(out.detach().norm())
    with torch.no_grad():
        for k, t in v.items():
            off = float((got[k].double() - t.grad).norm())
            assert off <= 5 * step * float(t.grad.norm()), (k, off / float(t.grad.norm()))
            d = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
            e = 1e-6
            diff = float(((output64({**v, k: t + e * d}, mod.EPS) - output64({**v, k: t - e * d}, mod.EPS)) * dy.double()).sum()) / (2 * e)
            assert abs(diff - float((t.grad * d).sum())) <= 1e-6 * float(t.grad.norm()) * float(d.norm()), k


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("width,hidden,rows", [(256, 688, 512), (72, 100, 130)])
def test_a_run_is_finite_and_the_same_twice(width, hidden, rows, bits):
    mod = load()
    first = mod.train(width, hidden, bits, steps=12, rows=rows)
    assert len(first) == 12 and all(math.isfinite(v) for v in first)
    assert mod.train(width, hidden, bits, steps=12, rows=rows) == first
