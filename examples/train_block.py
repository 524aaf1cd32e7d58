"""Train a pre-norm feed-forward block over W emulated data-parallel ranks with
the package's operators used together:

  - layer norm forward and backward (zero1_layernorm_*), the weight's and
    bias's gradients written straight into each rank's flat gradient buffer;
  - the matrix step (Muon) for the block's two matrices;
  - AdamW (Zero1) for the layer norm's vectors, at the end of the same flat
    buffers.

Everything lives in flat buffers: W bf16 gradients and replicas, one fp32
master and one fp32 momentum.  Matrices come first, vectors last, and the
AdamW handle is given the buffers from the vectors' offset on.

    python examples/train_block.py [--width 256] [--hidden 1024] [--world 4] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_adamw_gb300 as z  # noqa: E402

EPS = 1e-5


class Block:
    """y = x + relu(norm(x) W1) W2 for one rank: bf16 parameters and gradients
    are views of that rank's flat buffers."""

    def __init__(self, width: int, hidden: int, params: torch.Tensor, grads: torch.Tensor, rows: int):
        self.width, self.rows = width, rows
        sizes = [(width, hidden), (hidden, width), (width,), (width,)]
        self.p, self.g, at = [], [], 0
        for s in sizes:
            n = int(torch.tensor(s).prod())
            self.p.append(params[at:at + n].view(s))
            self.g.append(grads[at:at + n].view(s))
            at += n
        dev = params.device
        self.mean, self.rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        self.normed = torch.empty(rows, width, dtype=torch.bfloat16, device=dev)
        self.dx = torch.empty_like(self.normed)
        self.work = torch.empty(z.zero1_layernorm_workspace(rows, width), dtype=torch.uint8, device=dev)

    def step(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        """Forward, mean squared error, backward; gradients land in the flat buffer."""
        w1, w2, gamma, beta = self.p
        st = torch.cuda.current_stream()
        z.zero1_layernorm_forward(self.rows, self.width, z.DTYPE_BF16, x, self.width, gamma, beta, EPS, self.normed,
                                  self.width, self.mean, self.rstd, st)
        h = self.normed @ w1
        a = torch.relu(h)
        err = (x + a @ w2 - target).float()
        loss = err.square().mean()
        dy = (err * (2.0 / err.numel())).to(torch.bfloat16)
        torch.matmul(a.t(), dy, out=self.g[1])
        dh = (dy @ w2.t()) * (h > 0)
        torch.matmul(self.normed.t(), dh, out=self.g[0])
        dn = dh @ w1.t()
        z.zero1_layernorm_backward(self.rows, self.width, z.DTYPE_BF16, dn, self.width, x, self.width, gamma, self.mean,
                                   self.rstd, self.dx, self.width, self.g[2], self.g[3], z.DTYPE_BF16, self.work, st)
        return loss


def train(width: int = 256, hidden: int = 1024, world: int = 4, steps: int = 60, rows: int = 512, lr: float = 4e-3,
          seed: int = 0) -> list[float]:
    """Loss of every step (the mean over the ranks)."""
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    matrices = [(0, width, hidden), (width * hidden, hidden, width)]
    vectors = 2 * width * hidden
    n = vectors + 2 * width
    master = torch.empty(n, device=dev)
    master[:vectors].normal_(0.0, 0.02, generator=gen)
    master[vectors:vectors + width] = 1.0
    master[vectors + width:] = 0.0
    momentum = torch.zeros(n, device=dev)
    params = [master.to(torch.bfloat16) for _ in range(world)]
    grads = [torch.zeros(n, dtype=torch.bfloat16, device=dev) for _ in range(world)]
    blocks = [Block(width, hidden, p, g, rows) for p, g in zip(params, grads)]
    teacher = torch.randn(width, width, generator=gen, device=dev).mul_(width ** -0.5).to(torch.bfloat16)

    losses = []
    with z.Muon(n, world, matrices, z.MuonHparams(lr=lr, weight_decay=0.0)) as muon, \
            z.Zero1(2 * width, world, z.Hparams(lr=lr, weight_decay=0.0, max_norm=1.0)) as adam:
        adam.set_state(master[vectors:].contiguous())
        for _ in range(steps):
            total = torch.zeros((), device=dev)
            for b in blocks:                                   # each rank, its own data
                x = torch.randn(rows, width, generator=gen, device=dev).to(torch.bfloat16)
                total += b.step(x, x + torch.tanh(x @ teacher))
            st = torch.cuda.current_stream()
            muon.step(grads, params, master, momentum, st)
            adam.step([g[vectors:] for g in grads], [p[vectors:] for p in params], st)
            losses.append(total / world)
        muon.status()
        adam.grad_norm()
        return [float(v) for v in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--world", type=int, default=4)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.width, a.hidden, a.world, a.steps)):
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
