"""Measured cases of the matrix optimizer and of layer normalisation.

Four operators, each in a plain form (elementary torch operations in fp32,
rounded once at the end) and as this package's calls:

  orth    the Newton-Schulz orthogonalisation of each matrix of a flat buffer
          (zero1_muon_orthogonalize): X = U / (|U| + eps), then five times
          X = a X + (b A + c A A) X with A = X X^T (the smaller side's Gram
          matrix);
  step    one data-parallel step of the matrix optimizer built on it
          (zero1_muon_step): rank-ordered gradient mean, momentum, the
          orthogonalised update, decayed fp32 master, W bf16 replicas;
  ln_fwd  layer norm's forward pass (zero1_layernorm_forward);
  ln_bwd  its backward pass, with the weight's and bias's gradients summed
          over all rows (zero1_layernorm_backward).
"""
from __future__ import annotations

import math

import torch

own = False

# Coefficients of the quintic iteration, the number of steps, and the
# hyperparameters of a step (the learning rate, decay and master scale are
# those of this repository's workloads).
A, B, C, STEPS, EPS = 3.4445, -4.7750, 2.0315, 5, 1e-7
LR, MOMENTUM, DECAY, SCALE = 1e-3, 0.95, 0.1, 0.2
LN_EPS = 1e-5

# One transformer block's matrices of the GPT-2-small list, and the tiny
# workload's 4,096 parameters as one matrix.
BLOCK = "768x2304,768x768,768x3072,3072x768"
TINY = "64x64"


def listed():
    return [
        # The smallest call: one 4,096-entry matrix, all latency.
        {"name": "orth_tiny", "op": "orth", "shapes": TINY, "ld": 64, "dtype": "bf16"},
        # Odd sides, tall, padded rows, fp32 in and out.
        {"name": "orth_odd_f32", "op": "orth", "shapes": "1031x257,1031x257,1031x257", "ld": 263, "dtype": "f32"},
        # The query, key and value thirds of one fused 768 x 2304 gradient,
        # each orthogonalised by itself where it lies.
        {"name": "orth_qkv", "op": "orth", "shapes": "768x768,768x768,768x768", "ld": 2304, "slices": True,
         "dtype": "bf16"},
        # The largest: a feed-forward matrix of a 7B-class layer.
        {"name": "orth_large", "op": "orth", "shapes": "4096x16384", "ld": 16384, "dtype": "bf16"},
        # A whole step at the tiny workload's size and ranks.
        {"name": "step_tiny", "op": "step", "shapes": TINY, "world": 4},
        # One GPT-2-small block, W = 8: a step run layer by layer.
        {"name": "step_block", "op": "step", "shapes": BLOCK, "world": 8},
        # All twelve blocks, W = 8: the whole model's matrices.
        {"name": "step_gpt2", "op": "step", "shapes": ",".join([BLOCK] * 12), "world": 8},
        # One token while serving.
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 768, "pad": 0, "dtype": "bf16"},
        # A training batch of 16 sequences of 1,024 tokens.
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 16384, "cols": 768, "pad": 0, "dtype": "bf16"},
        # The same batch backwards.
        {"name": "ln_bwd_batch", "op": "ln_bwd", "rows": 16384, "cols": 768, "pad": 0, "dtype": "bf16"},
        # Odd rows and columns in fp32, rows that start off any alignment.
        {"name": "ln_bwd_odd_f32", "op": "ln_bwd", "rows": 1003, "cols": 1021, "pad": 2, "dtype": "f32"},
        # A large model's batch: 65,536 tokens of width 4,096.
        {"name": "ln_bwd_large", "op": "ln_bwd", "rows": 65536, "cols": 4096, "pad": 0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["orth", "step", "ln_fwd", "ln_bwd"])
    if op == "orth":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        # fp32 updates are asked for where matrices are small
        rows, cols = (_log(rng, 16, 4096 if dtype == "bf16" else 1200) for _ in range(2))
        count = _log(rng, 1, 12) if max(rows, cols) <= 1500 else 1
        return {"op": op, "shapes": ",".join(["%dx%d" % (rows, cols)] * count), "ld": cols + rng.choice([0, 0, 1, 8, 37]),
                "dtype": dtype}
    if op == "step":
        shapes = ",".join("%dx%d" % (_log(rng, 24, 2304), _log(rng, 24, 2304)) for _ in range(_log(rng, 1, 8)))
        return {"op": op, "shapes": shapes, "world": _log(rng, 1, 16)}
    cols = _log(rng, 16, 8192)
    rows = _log(rng, 1, min(65536, (1 << 26) // cols))
    return {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 0, 1, 8, 13]),
            "dtype": rng.choice(["bf16", "f32"])}


# ----------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _layout(case):
    """[(offset, rows, cols, ld)] of the matrices in their flat buffer, and its length."""
    out, at = [], 0
    for i, (r, c) in enumerate(_shapes(case)):
        if case.get("slices"):
            out.append((i * c, r, c, case["ld"]))
            at = r * case["ld"]
        else:
            ld = case.get("ld", c)
            out.append((at, r, c, ld))
            at += r * ld
    return out, at


def _view(flat, m):
    off, r, c, ld = m
    return torch.as_strided(flat, (r, c), (ld, 1), flat.storage_offset() + off)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": dict(case)}
    if case["op"] in ("orth", "step"):
        mats, n = _layout(case)
        s["mats"], s["n"] = mats, n

        def gradient(scale):
            # noise over a few strong directions, as gradients of matrices have
            flat = randn(n).mul_(scale)
            for m in mats:
                v = _view(flat, m)
                k = max(1, min(8, m[1] // 4, m[2] // 4))
                v.add_(randn(m[1], k) @ randn(k, m[2]), alpha=scale / math.sqrt(k))
            return flat

        if case["op"] == "orth":
            s["u"] = gradient(1e-3).to(_DT[case["dtype"]])
            s["out"] = torch.zeros(n, dtype=_DT[case["dtype"]], device="cuda")
        else:
            w = case["world"]
            common = gradient(1e-3)
            s["grads"] = [(common + randn(n).mul_(1e-3)).to(torch.bfloat16) for _ in range(w)]
            s["params"] = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(w)]
            s["master"] = randn(n).mul_(0.02)
            s["momentum"] = gradient(5e-4)
    else:
        rows, cols, dt = case["rows"], case["cols"], _DT[case["dtype"]]

        def activations(scale, shift):
            full = torch.empty(rows, cols + case["pad"], dtype=dt, device="cuda")
            full.copy_(randn(rows, cols + case["pad"]).mul_(scale).add_(shift))
            return full[:, :cols]

        s["x"] = activations(1.5, 0.3)
        s["gamma"] = (1 + 0.1 * randn(cols)).to(dt)
        s["beta"] = (0.1 * randn(cols)).to(dt)
        if case["op"] == "ln_bwd":
            s["dy"] = activations(1e-2, 0.0)
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square_().mean(1) + LN_EPS).rsqrt().float()
            s["dx"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            s["dgamma"], s["dbeta"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        else:
            s["y"] = torch.empty(rows, cols, dtype=dt, device="cuda")
            s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import zero_sharded_adamw_gb300 as z
        if case["op"] in ("orth", "step"):
            hp = z.MuonHparams(lr=LR, momentum=MOMENTUM, weight_decay=DECAY, eps=EPS, update_scale=SCALE,
                               ns_steps=STEPS, ns_a=A, ns_b=B, ns_c=C)
            s["opt"] = z.Muon(s["n"], case.get("world", 1), s["mats"], hp)
        elif case["op"] == "ln_bwd":
            s["workspace"] = torch.empty(z.zero1_layernorm_workspace(case["rows"], case["cols"]), dtype=torch.uint8,
                                         device="cuda")
    return s


# -------------------------------------------------------------- one pass

def _orthogonal(u):
    """The plain form of the iteration on one fp32 matrix."""
    x = u.t() if u.shape[0] > u.shape[1] else u
    x = x / (x.square().sum().sqrt() + EPS)
    for _ in range(STEPS):
        a = x @ x.t()
        x = A * x + (B * a + C * (a @ a)) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def _plain_orth(s):
    out = torch.zeros_like(s["u"])
    for m in s["mats"]:
        _view(out, m).copy_(_orthogonal(_view(s["u"], m).float()))
    return {"out": out}


def _plain_step(s):
    total = s["grads"][0].float()
    for g in s["grads"][1:]:
        total = total + g.float()
    mean = total * (1.0 / len(s["grads"]))
    s["momentum"].copy_(MOMENTUM * s["momentum"] + (1 - MOMENTUM) * mean)
    u = MOMENTUM * s["momentum"] + (1 - MOMENTUM) * mean
    for m in s["mats"]:
        p = _view(s["master"], m)
        p.copy_(p * (1 - LR * DECAY) - (LR * SCALE * math.sqrt(max(m[1], m[2]))) * _orthogonal(_view(u, m)))
    low = s["master"].to(torch.bfloat16)
    for q in s["params"]:
        q.copy_(low)
    return {"params": s["params"], "master": s["master"], "momentum": s["momentum"]}


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / (d.square().mean(1, keepdim=True) + LN_EPS).sqrt()
    y = d * rstd * s["gamma"].float() + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_ln_bwd(s):
    rstd = s["rstd"][:, None]
    h = (s["x"].float() - s["mean"][:, None]) * rstd
    dy = s["dy"].float()
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"orth": _plain_orth, "step": _plain_step, "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}[op](s)
    import zero_sharded_adamw_gb300 as z
    stream = torch.cuda.current_stream()
    if op == "orth":
        s["opt"].orthogonalize(s["u"], s["out"], stream)
        return {"out": s["out"]}
    if op == "step":
        s["opt"].step(s["grads"], s["params"], s["master"], s["momentum"], stream)
        return {"params": s["params"], "master": s["master"], "momentum": s["momentum"]}
    x = s["x"]
    rows, cols = x.shape
    dtype = z.DTYPE_BF16 if x.dtype == torch.bfloat16 else z.DTYPE_F32
    if op == "ln_fwd":
        z.zero1_layernorm_forward(rows, cols, dtype, x, x.stride(0), s["gamma"], s["beta"], LN_EPS, s["y"],
                                  s["y"].stride(0), s["mean"], s["rstd"], stream)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    z.zero1_layernorm_backward(rows, cols, dtype, s["dy"], s["dy"].stride(0), x, x.stride(0), s["gamma"], s["mean"],
                               s["rstd"], s["dx"], s["dx"].stride(0), s["dgamma"], s["dbeta"], z.DTYPE_F32,
                               s["workspace"], stream)
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


# ------------------------------------------------------------------ work

def work(case):
    """Each input read once, each output written once; for the iteration the
    Gram matrix and its square as the symmetric matrices they are (s*s*l and
    s*s*s operations for sides s <= l) and the product with X (2*s*s*l)."""
    if case["op"] in ("orth", "step"):
        entries = sum(r * c for r, c in _shapes(case))
        flops = 0
        for r, c in _shapes(case):
            s, l = min(r, c), max(r, c)
            flops += STEPS * (3 * s * s * l + s * s * s)
        if case["op"] == "orth":
            return {"bytes": entries * 2 * (2 if case["dtype"] == "bf16" else 4), "flops": flops}
        # W gradients in, W replicas out, master and momentum in and out
        return {"bytes": entries * (4 * case["world"] + 16), "flops": flops}
    e = 2 if case["dtype"] == "bf16" else 4
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * rows * cols * e + 2 * cols * e + 8 * rows, "flops": 8 * rows * cols}
    return {"bytes": 3 * rows * cols * e + cols * e + 8 * rows + 8 * cols, "flops": 14 * rows * cols}


# ----------------------------------------------------------------- exact

def _orthogonal64(u):
    """The iteration in 64 bits through the Gram matrix alone: with G = X X^T
    and X' = P X, G' = P G P, so the product R of the P's is gathered and
    applied once."""
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    gram, r = x @ x.t(), eye
    for _ in range(STEPS):
        p = A * eye + gram @ (B * eye + C * gram)
        r = p @ r
        gram = p @ gram @ p
    x = r @ x
    return x.t() if tall else x


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "orth":
        out = torch.zeros(s["n"], dtype=torch.float64, device="cuda")
        for m in s["mats"]:
            _view(out, m).copy_(_orthogonal64(_view(s["u"], m)))
        return {"out": out}
    if case["op"] == "step":
        mean = torch.stack([g.double() for g in s["grads"]]).mean(0) if s["n"] < 1 << 24 else \
            sum(g.double() for g in s["grads"]) / len(s["grads"])
        momentum = s["momentum"].double() * MOMENTUM + mean * (1 - MOMENTUM)
        master = s["master"].double()
        look_ahead = momentum * MOMENTUM + mean * (1 - MOMENTUM)
        for m in s["mats"]:
            p = _view(master, m)
            p.mul_(1 - LR * DECAY).sub_(_orthogonal64(_view(look_ahead, m)),
                                        alpha=LR * SCALE * max(m[1], m[2]) ** 0.5)
        return {"params": [master] * len(s["params"]), "master": master, "momentum": momentum}
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["op"] == "ln_fwd":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = (var + LN_EPS).pow(-0.5)
        return {"y": torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma), "mean": mean,
                "rstd": rstd}
    dy, mean, rstd = s["dy"].double(), s["mean"].double(), s["rstd"].double()
    n = x.shape[1]
    hat = (x - mean[:, None]).mul_(rstd[:, None])
    del x
    dgamma, dbeta = torch.einsum("ij,ij->j", dy, hat), dy.sum(0)
    dy.mul_(gamma)
    dx = dy - (dy.sum(1) / n)[:, None] - hat * (torch.einsum("ij,ij->i", dy, hat) / n)[:, None]
    return {"dx": dx.mul_(rstd[:, None]), "dgamma": dgamma, "dbeta": dbeta}
