"""The AdamW step over many tensors as its documentation writes it, in plain
torch operations: every fp32 operation by itself, and a step in 64 bits."""
from __future__ import annotations

import math

import torch

BLOCK = 256
M_TOP, R_TOP = 61439.0, 63487.0


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def starts(sizes) -> tuple[list[int], int]:
    out, at = [], 0
    for n in sizes:
        out.append(at)
        at += blocks(n) * BLOCK
    return out, at


def mix(x):
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def dither(n: int, seed: int, t: int, device):
    """Two 16-bit numbers an entry (places below 2^32)."""
    key = mix(mix(mix(seed & 0xFFFFFFFF) ^ (seed >> 32)) ^ (t & 0xFFFFFFFF))
    h = mix(torch.arange(n, device=device) ^ key)
    return h & 0xFFFF, h >> 16


def value(k, bits: int):
    """f(k, bits) - 1, exact in any type."""
    k = k.double()
    octave = torch.floor(k / 2 ** bits)
    return torch.exp2(octave) * (1 + (k - octave * 2 ** bits) / 2 ** bits) - 1


def decode(km, kr, scales):
    """m and sqrt(v) as fp32: one product each."""
    sm, sr = (scales[:, i].repeat_interleave(BLOCK) for i in (0, 1))
    mag = value(km & 127, 3).float() * sm
    return torch.where(km >= 128, -mag, mag), value(kr, 4).float() * sr


def encode(x, top: float, bits: int, random16, keep: bool):
    """Codes of |x| and block scales; keep: what is not zero gets no zero code."""
    x = x.abs().view(-1, BLOCK)
    most = torch.where(x.isnan().any(1), torch.full_like(x[:, 0], math.nan), x.amax(1))
    held = (most >= 2.0 ** -100) & (most < math.inf)
    tops = torch.full_like(most, top)
    scale = torch.where(held, most / tops, torch.where(most < 2.0 ** -100, most * 0, most * math.nan))
    inv = torch.where(held, tops / most, most.new_zeros(()))
    y = (x * inv[:, None] + 1.0).view(torch.int32).long() + (random16.view(-1, BLOCK) << (7 - bits))
    k = ((y - (127 << 23)) >> (23 - bits)).clamp(0, 16 * 2 ** bits - 1)
    if keep:
        k = torch.where((k == 0) & (x > 0), torch.ones_like(k), k)
    return torch.where(held[:, None], k, torch.zeros_like(k)).view(-1), scale


def scalars(hp, t: int):
    """lr sqrt(1-beta2^t)/(1-beta1^t) and 1 - lr wd, as Python doubles."""
    return hp.lr * (math.sqrt(1.0 - hp.beta2 ** t) / (1.0 - hp.beta1 ** t)), 1.0 - hp.lr * hp.weight_decay


def step(g, w, m, v, hp, t: int, decays, clip, decay_first=False):
    """One step of flat fp32 tensors (g unclipped; `clip` an fp32 scalar tensor
    or None; `decays` a truth value an entry): new w, m, v."""
    size, keep = scalars(hp, t)
    if clip is not None:
        g = g * clip
    m = hp.beta1 * m + (1.0 - hp.beta1) * g
    v = hp.beta2 * v + ((1.0 - hp.beta2) * g) * g
    u = size * (m / (v.sqrt() + hp.eps))
    if decay_first:
        w = torch.where(decays, w * keep, w)
    w = w - u
    if not decay_first:
        w = torch.where(decays, w * keep, w)
    return w, m, v
