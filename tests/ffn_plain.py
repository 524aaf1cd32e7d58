"""The gated feed-forward block in 64 bits, with bounds on how far results in
bf16 with fp32 sums may be from it."""
from __future__ import annotations

import math

import torch

E = 2.0 ** -8        # a bf16 rounding: half a step, relative
SUM = 2.0 ** -23     # what an fp32 addition that cuts off may lose, relative to the sum of magnitudes so far
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def act(g, name):
    """The activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    return torch.where(g <= 0, torch.zeros_like(g), g), (g > 0).to(g.dtype)


def product(a, b, da=None):
    """a b, and how far it may be off: one addition cut off for each 8 of K
    (the tensor cores add 16 products at a time) relative to the sum of
    magnitudes, and the error `da` of a."""
    size = a.abs() @ b.abs()
    off = (a.shape[1] / 8 + 2) * SUM * size
    return a @ b, off if da is None else off + da @ b.abs()


def forward(x, wg, wu, wd, name):
    """{name: (value, bound)} of gate, up, h and y as bf16."""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    gate, dg = product(x, wg)
    up, du = product(x, wu)
    a, _ = act(gate, name)
    h = a * up
    # |act'| <= 1.13; the activation in fp32: 1e-5 of |g| at most (erf near -1, the approximate exponential)
    dh = 1.13 * dg * up.abs() + a.abs() * du + dg * du * 1.13 + 1e-5 * gate.abs() * up.abs()
    h_off = dh + (h.abs() + dh) * E
    y, dy = product(h, wd, h_off)
    low = lambda v, d: (v, d + (v.abs() + d) * E + 1e-37)  # noqa: E731
    return {"gate": low(gate, dg), "up": low(up, du), "h": (h, h_off + 1e-37), "y": low(y, dy)}


def backward(dy, x, wg, wu, wd, gate, up, h, name):
    """{name: (value, bound)} of dx, dw_gate, dw_up and dw_down as bf16."""
    dy, x, wg, wu, wd, gate, up, h = (t.double() for t in (dy, x, wg, wu, wd, gate, up, h))
    dh, d = product(dy, wd.t())
    a, slope = act(gate, name)
    dgate, dup = dh * up * slope, dh * a
    slack = 1e-5 * (1 + gate.abs())
    off_g = d * (up * slope).abs() + dh.abs() * up.abs() * slack
    off_u = d * a.abs() + dh.abs() * gate.abs() * slack
    off_g, off_u = off_g + (dgate.abs() + off_g) * E, off_u + (dup.abs() + off_u) * E
    dx1, e1 = product(dgate, wg.t(), off_g)
    dx2, e2 = product(dup, wu.t(), off_u)
    # one sum over both: its additions are relative to both magnitudes
    both = (dgate.abs() @ wg.abs().t() + dup.abs() @ wu.abs().t()) * (2 * gate.shape[1] / 8 + 2) * SUM
    rows = x.shape[0]

    def weight(left, right, off):
        size = left.abs().t() @ right.abs()
        return left.t() @ right, (rows / 8 + 2) * SUM * size + left.abs().t() @ off

    low = lambda v, d: (v, d + (v.abs() + d) * E + 1e-37)  # noqa: E731
    return {"dx": low(dx1 + dx2, e1 + e2 + both), "dw_gate": low(*weight(x, dgate, off_g)),
            "dw_up": low(*weight(x, dup, off_u)), "dw_down": low(*weight(h, dy, torch.zeros_like(dy)))}
