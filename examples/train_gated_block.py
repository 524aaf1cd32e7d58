"""Train a pre-norm gated feed-forward block, y = x + W_down (silu(n W_gate) *
(n W_up)) with n = norm(x), whose parameters are a list of tensors:

  - layer norm forward and backward (zero1_layernorm_*);
  - the gated feed-forward block forward and backward (zero1_ffn_*);
  - AdamW over the list (zero1_adamw_*), its moments in 32 or 8 bits, the
    vectors spared the weight decay.

    python examples/train_gated_block.py [--width 256] [--hidden 688] [--bits 8] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_adamw_gb300 as z  # noqa: E402

EPS = 1e-5
NAMES = ("w_gate", "w_up", "w_down", "gamma", "beta")


class GatedBlock:
    """The block for batches of `rows` rows: parameters `p` and gradients `g`
    by name, and the activations between forward and backward."""

    def __init__(self, width: int, hidden: int, rows: int, generator: torch.Generator):
        dev = generator.device

        def bf16(*shape):
            return torch.empty(*shape, dtype=torch.bfloat16, device=dev)

        shapes = dict(w_gate=(width, hidden), w_up=(width, hidden), w_down=(hidden, width), gamma=(width,), beta=(width,))
        self.p = {k: bf16(*s) for k, s in shapes.items()}
        self.g = {k: torch.zeros_like(v) for k, v in self.p.items()}
        for k in NAMES[:3]:
            self.p[k].copy_(torch.randn(shapes[k], generator=generator, device=dev) * shapes[k][0] ** -0.5)
        self.p["gamma"].fill_(1.0)
        self.p["beta"].zero_()
        self.rows, self.width = rows, width
        self.shape = z.FfnShape(rows, width, hidden, z.ACT_SILU)
        self.mean, self.rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        self.n, self.y, self.dn, self.dx = (bf16(rows, width) for _ in range(4))
        self.gate, self.up, self.h = (bf16(rows, hidden) for _ in range(3))
        self.work = torch.empty(max(z.zero1_ffn_workspace(self.shape, True), z.zero1_ffn_workspace(self.shape),
                                    z.zero1_layernorm_workspace(rows, width)), dtype=torch.uint8, device=dev)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        st, p, w = torch.cuda.current_stream(), self.p, self.width
        z.zero1_layernorm_forward(self.rows, w, z.DTYPE_BF16, x, w, p["gamma"], p["beta"], EPS, self.n, w, self.mean,
                                  self.rstd, st)
        z.zero1_ffn_forward(self.shape, self.n, p["w_gate"], p["w_up"], p["w_down"], self.gate, self.up, self.h, self.y,
                            self.work, st)
        return x + self.y

    def backward(self, x: torch.Tensor, dy: torch.Tensor) -> torch.Tensor:
        """Gradients of the parameters into `g`; returns that of x."""
        st, p, g, w = torch.cuda.current_stream(), self.p, self.g, self.width
        z.zero1_ffn_backward(self.shape, dy, self.n, p["w_gate"], p["w_up"], p["w_down"], self.gate, self.up, self.h,
                             self.dn, g["w_gate"], g["w_up"], g["w_down"], self.work, st)
        z.zero1_layernorm_backward(self.rows, w, z.DTYPE_BF16, self.dn, w, x, w, p["gamma"], self.mean, self.rstd,
                                   self.dx, w, g["gamma"], g["beta"], z.DTYPE_BF16, self.work, st)
        return self.dx + dy


def train(width: int = 256, hidden: int = 688, bits: int = 8, steps: int = 60, rows: int = 512, lr: float = 3e-3,
          seed: int = 0) -> list[float]:
    """Loss of every step."""
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    block = GatedBlock(width, hidden, rows, gen)
    params, grads = [block.p[k] for k in NAMES], [block.g[k] for k in NAMES]
    teacher = torch.randn(width, width, generator=gen, device=dev).mul_(width ** -0.5)
    losses = []
    with z.AdamW([t.numel() for t in params], z.Hparams(lr=lr, max_norm=1.0), z.AdamWOptions(state_bits=bits, seed=seed),
                 decays=[t.dim() > 1 for t in params]) as opt:
        # the state: one buffer each, a tensor's part from opt.starts on
        kind = torch.uint8 if bits == 8 else torch.float32
        master = torch.zeros(opt.entries, device=dev)
        for t, at in zip(params, opt.starts):
            master[at:at + t.numel()] = t.float().view(-1)
        m, v = torch.zeros(opt.entries, dtype=kind, device=dev), torch.zeros(opt.entries, dtype=kind, device=dev)
        scales = torch.zeros(opt.scale_entries, device=dev) if bits == 8 else None
        tables = z.PtrTable(grads), z.PtrTable(params)
        for _ in range(steps):
            x = torch.randn(rows, width, generator=gen, device=dev).to(torch.bfloat16)
            target = x + torch.tanh(x.float() @ teacher)
            err = block.forward(x).float() - target
            block.backward(x, (err * (2.0 / err.numel())).to(torch.bfloat16))
            opt.step(*tables, master, m, v, scales, torch.cuda.current_stream())
            losses.append(err.square().mean())
        opt.grad_norm()
        return [float(x) for x in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=688)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.width, a.hidden, a.bits, a.steps)):
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
