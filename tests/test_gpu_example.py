"""The example that uses the matrix step, layer norm and AdamW together: it
learns as the same training in plain torch operations does, and gives the
same losses every time."""
from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def orth(u):
    x = u.t() if u.shape[0] > u.shape[1] else u
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        a = x @ x.t()
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * (a @ a)) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def plain(width, hidden, world, steps, rows, lr=4e-3):
    """The same training in fp32: autograd, momentum and orthogonalised update
    for the matrices, clipped AdamW for the vectors."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = 2 * width * hidden
    flat = torch.empty(n + 2 * width, device="cuda")
    flat[:n].normal_(0.0, 0.02, generator=gen)
    teacher = torch.randn(width, width, generator=gen, device="cuda").mul_(width ** -0.5).to(torch.bfloat16)
    mats = [flat[:n // 2].view(width, hidden).clone(), flat[n // 2:n].view(hidden, width).clone()]
    vec = torch.cat([torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")])
    mom = [torch.zeros_like(m) for m in mats]
    m1, m2, losses = torch.zeros_like(vec), torch.zeros_like(vec), []
    for t in range(1, steps + 1):
        leaves = [p.clone().requires_grad_() for p in (*mats, vec)]
        total = 0.0
        for _ in range(world):
            x = torch.randn(rows, width, generator=gen, device="cuda").to(torch.bfloat16)
            target = (x + torch.tanh(x @ teacher)).float()
            x = x.float()
            h = torch.nn.functional.layer_norm(x, (width,), leaves[2][:width], leaves[2][width:], 1e-5)
            total = total + (x + torch.relu(h @ leaves[0]) @ leaves[1] - target).square().mean()
        (total / world).backward()
        losses.append(float(total.detach()) / world)
        for p, m, leaf in zip(mats, mom, leaves):
            m.mul_(0.95).add_(leaf.grad, alpha=0.05)
            p.sub_(orth(0.95 * m + 0.05 * leaf.grad), alpha=lr * 0.2 * math.sqrt(max(p.shape)))
        g = leaves[2].grad
        g = g * min(1.0, 1.0 / float(g.norm()))
        m1.mul_(0.9).add_(g, alpha=0.1)
        m2.mul_(0.95).add_(g * g, alpha=0.05)
        vec.sub_(m1 / (m2.sqrt() + 1e-8), alpha=lr * math.sqrt(1 - 0.95 ** t) / (1 - 0.9 ** t))
    return losses


@pytest.mark.parametrize("width,hidden,world", [(256, 1024, 4), (64, 96, 2), (136, 200, 3)])
def test_example_learns_as_plain_training_does(width, hidden, world):
    """Parameters, activations and gradients of the example are bf16.  A
    rounding is 2^-9 of an entry at random, and the orthogonalised update
    gives the gradient's weakest directions, where that counts most, as much
    weight as its strongest, so the two paths part slowly; both descend the
    same loss, whose values are means over 16,000 and more entries.  They stay
    within 5% of each other while the loss falls by a third and more."""
    mod = load()
    first = mod.train(width, hidden, world, steps=60, rows=256)
    want = plain(width, hidden, world, 60, 256)
    assert all(abs(a - b) <= 0.05 * b for a, b in zip(first, want)), (first[-1], want[-1])
    assert first[-1] < 0.7 * first[0]
    assert mod.train(width, hidden, world, steps=60, rows=256) == first
