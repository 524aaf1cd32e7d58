"""Measured cases of the AdamW step over a list of tensors and of the gated
feed-forward block.

Three operators, each in a plain form (elementary torch operations in fp32,
rounded once at the end) and as this package's calls:

  adamw    one AdamW step over many tensors at once (zero1_adamw_step), its
           moments held in 32 bits, or in 8 bits with two scales for each
           block of 256 entries.  With 8 bits a pass also reads the moments
           out as the values they stand for (zero1_adamw_moments);
  ffn_fwd  y = (act(x Wg) * (x Wu)) Wd, keeping h = act(x Wg) * (x Wu) and, for
           training, both projections (zero1_ffn_forward);
  ffn_bwd  its gradients for x and the three matrices (zero1_ffn_backward).

The 8-bit codes, of entries of a block whose largest |m| is M and whose
largest sqrt(v) is R: with f(k, b) = (1 + (k mod 2^b)/2^b) 2^(k div 2^b),

  m       = +-(f(k, 3) - 1) * (M / 61439),   k of 7 bits beside the sign,
  sqrt(v) =   (f(k, 4) - 1) * (R / 63487),   k of 8 bits,

rounded up or down at random by 16 bits each of a hash of the seed, the step
and the entry's place, so that the expected value is the exact one.
"""
from __future__ import annotations

import math

import torch

own = False

# Hyperparameters of this repository's workloads; the states are those after
# ten steps.
LR, BETA1, BETA2, ADAM_EPS, DECAY, MAX_NORM, STEPS_DONE, SEED = 1e-3, 0.9, 0.95, 1e-8, 0.1, 1.0, 10, 1234

# The GPT-2-small parameter list of this repository's workloads as "rows x cols" and vectors.
GPT2 = "50257x768,1024x768," + ",".join(["768x2304,768x768,768x3072,3072x768,768,768,768,768"] * 12)
# A layer of width 4096 with a gated feed-forward block (hidden 11008: two
# thirds of four times the width, rounded up to 256).
LAYER = "4096x4096,4096x4096,4096x4096,4096x4096,4096x11008,4096x11008,11008x4096,4096,4096"


def listed():
    return [
        # The tiny workload's 4,096 parameters: a matrix and its bias, all latency.
        {"name": "adamw_tiny", "op": "adamw", "tensors": "64x63,64", "bits": 32, "dtype": "bf16", "clip": True,
         "packed": False},
        # The GPT-2-small list, 98 tensors, clipped: the whole model's step.
        {"name": "adamw_gpt2", "op": "adamw", "tensors": GPT2, "bits": 32, "dtype": "bf16", "clip": True,
         "packed": False},
        # The same with moments in 8 bits.
        {"name": "adamw8_gpt2", "op": "adamw", "tensors": GPT2, "bits": 8, "dtype": "bf16", "clip": True,
         "packed": False},
        # fp32 parameters and gradients of odd sizes, packed one after another
        # without alignment, not clipped.
        {"name": "adamw8_odd_f32", "op": "adamw", "tensors": "1021x513,513,1,77x1021,255,1003x1001,257", "bits": 8,
         "dtype": "f32", "clip": False, "packed": True},
        # Two layers of width 4096: the step where memory counts most.
        {"name": "adamw8_large", "op": "adamw", "tensors": LAYER + "," + LAYER, "bits": 8, "dtype": "bf16",
         "clip": True, "packed": False},
        # One token while serving a model of width 768.
        {"name": "ffn_fwd_token", "op": "ffn_fwd", "rows": 1, "width": 768, "hidden": 2048, "pad": 0, "act": "silu",
         "train": False},
        # Eight sequences' next tokens at width 4096: the weights are what is read.
        {"name": "ffn_fwd_decode", "op": "ffn_fwd", "rows": 8, "width": 4096, "hidden": 11008, "pad": 0,
         "act": "silu", "train": False},
        # A ragged prompt with odd widths and rows off any alignment.
        {"name": "ffn_fwd_odd", "op": "ffn_fwd", "rows": 1003, "width": 517, "hidden": 1365, "pad": 2, "act": "gelu",
         "train": True},
        # A training batch of 16 sequences of 1,024 tokens.
        {"name": "ffn_fwd_batch", "op": "ffn_fwd", "rows": 16384, "width": 768, "hidden": 2048, "pad": 0,
         "act": "silu", "train": True},
        # A small batch backwards: few tiles, a long sum over rows.
        {"name": "ffn_bwd_small", "op": "ffn_bwd", "rows": 2000, "width": 256, "hidden": 688, "pad": 0, "act": "gelu",
         "train": True},
        # The training batch backwards.
        {"name": "ffn_bwd_batch", "op": "ffn_bwd", "rows": 16384, "width": 768, "hidden": 2048, "pad": 0,
         "act": "silu", "train": True},
        # A large model's batch backwards: 8,192 tokens of width 4096.
        {"name": "ffn_bwd_large", "op": "ffn_bwd", "rows": 8192, "width": 4096, "hidden": 11008, "pad": 0,
         "act": "silu", "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "ffn_fwd", "ffn_bwd"])
    if op == "adamw":
        left, shapes = _log(rng, 1 << 10, 1 << 27), []
        for _ in range(_log(rng, 1, 160)):
            n = min(left, _log(rng, 1, max(2, left // 2)))
            cols = min(n, _log(rng, 1, 4096))
            shapes.append("%dx%d" % (max(1, n // cols), cols) if rng.random() < 0.7 else str(n))
            left = max(1, left - n)
        return {"op": op, "tensors": ",".join(shapes), "bits": rng.choice([8, 32]), "dtype": rng.choice(["bf16", "f32"]),
                "clip": rng.random() < 0.5, "packed": rng.random() < 0.3}
    width, hidden = _log(rng, 16, 4096), _log(rng, 16, 11008)
    rows = _log(rng, 1, max(16, min(16384, (1 << 38) // (width * hidden))))
    return {"op": op, "rows": rows, "width": width, "hidden": hidden, "pad": rng.choice([0, 0, 0, 1, 8, 13]),
            "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), "train": op == "ffn_bwd" or rng.random() < 0.5}


# ----------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK, M_TOP, R_TOP, M_BITS, R_BITS = 256, 61439.0, 63487.0, 3, 4
TINY = 2.0 ** -100      # a block whose largest value is smaller is held as zeros


def _sizes(case):
    return [math.prod(int(v) for v in t.split("x")) for t in case["tensors"].split(",")]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "adamw":
        sizes, dt = _sizes(case), _DT[case["dtype"]]
        # where each tensor's state lies: whole blocks
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += -(-n // BLOCK) * BLOCK
        s["spans"], s["n"], s["t"] = [(a, a + n) for a, n in zip(starts, sizes)], at, STEPS_DONE

        # parameters and gradients: views of one allocation each, aligned as
        # separate allocations are, or packed without gaps
        def tensors(flat):
            if case["packed"]:
                low = torch.cat([flat[a:b] for a, b in s["spans"]]).to(dt)
                return low, list(low.split(sizes))
            low = flat.to(dt)
            return low, [low[a:b] for a, b in s["spans"]]

        held = torch.zeros(at, device="cuda")
        for a, b in s["spans"]:
            held[a:b] = 1.0
        # gradients and moments of unlike magnitude from row to row, as those
        # of embeddings and early layers are
        scale = held * torch.exp(0.7 * randn(at // 64 + 1)).repeat_interleave(64)[:at] * 1e-3
        master = randn(at).mul_(0.02).mul_(held)
        s["grad_flat"], s["grads"] = tensors(randn(at).mul_(scale))
        s["param_flat"], s["params"] = tensors(master)
        s["master"] = master if case["dtype"] == "bf16" else None
        m = randn(at).mul_(scale).mul_(0.3)
        v = scale.square_().mul_(0.4).mul_(0.5 + torch.rand(at, generator=g, device="cuda"))
        if case["bits"] == 32:
            s["m"], s["v"], s["scales"] = m, v, None
        else:
            half = torch.full((at,), 0x8000, dtype=torch.int32, device="cuda")
            s["m"], ms = _encode(m, m < 0, M_TOP, M_BITS, half)
            s["v"], vs = _encode(v.sqrt(), None, R_TOP, R_BITS, half)
            s["scales"] = torch.stack([ms, vs], 1).contiguous()
            s["m_out"], s["v_out"] = torch.zeros(at, device="cuda"), torch.zeros(at, device="cuda")
    else:
        rows, width, hidden, pad = case["rows"], case["width"], case["hidden"], case["pad"]

        def matrix(r, c, scale, shift=0.0):
            full = torch.empty(r, c + pad, dtype=torch.bfloat16, device="cuda")
            full.copy_(randn(r, c + pad).mul_(scale).add_(shift))
            return full[:, :c]

        s["x"] = matrix(rows, width, 1.0, 0.1)
        s["w_gate"], s["w_up"] = matrix(width, hidden, width ** -0.5), matrix(width, hidden, width ** -0.5)
        s["w_down"] = matrix(hidden, width, hidden ** -0.5)
        if case["op"] == "ffn_fwd":
            if case["train"]:
                s["gate"], s["up"] = matrix(rows, hidden, 0.0), matrix(rows, hidden, 0.0)
            s["h"], s["y"] = matrix(rows, hidden, 0.0), matrix(rows, width, 0.0)
        else:
            s["gate"], s["up"] = matrix(rows, hidden, 1.0), matrix(rows, hidden, 1.0)
            s["h"] = matrix(rows, hidden, 0.0)
            s["h"].copy_(_act(s["gate"].float(), case["act"]) * s["up"].float())
            s["dy"] = matrix(rows, width, 1e-2)
            s["dx"] = matrix(rows, width, 0.0)
            s["dw_gate"], s["dw_up"] = matrix(width, hidden, 0.0), matrix(width, hidden, 0.0)
            s["dw_down"] = matrix(hidden, width, 0.0)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import zero_sharded_adamw_gb300 as z
        if case["op"] == "adamw":
            dtype = z.DTYPE_BF16 if case["dtype"] == "bf16" else z.DTYPE_F32
            hp = z.Hparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY,
                           max_norm=MAX_NORM if case["clip"] else 0.0)
            s["opt"] = z.AdamW(_sizes(case), hp, z.AdamWOptions(state_bits=case["bits"], param_dtype=dtype,
                                                               grad_dtype=dtype, seed=SEED))
            s["opt"].set_steps(STEPS_DONE, torch.cuda.current_stream())
            s["grad_table"], s["param_table"] = z.PtrTable(s["grads"]), z.PtrTable(s["params"])
        else:
            act = {"silu": z.ACT_SILU, "gelu": z.ACT_GELU, "gelu_tanh": z.ACT_GELU_TANH, "relu": z.ACT_RELU}
            rows, width, hidden, pad = case["rows"], case["width"], case["hidden"], case["pad"]
            s["shape"] = z.FfnShape(rows, width, hidden, act[case["act"]], ldx=width + pad, ldy=width + pad,
                                    ldh=hidden + pad, ld_gate=hidden + pad, ld_up=hidden + pad, ld_down=width + pad)
            s["workspace"] = torch.empty(z.zero1_ffn_workspace(s["shape"], case["op"] == "ffn_bwd"),
                                         dtype=torch.uint8, device="cuda")
    return s


# -------------------------------------------------------------- one pass

def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return sig * (1.0 + g * (1.0 - sig))
    if act == "relu":
        return (g > 0).to(g.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * math.sqrt(2 / math.pi) * (1.0 + 3 * 0.044715 * g * g)


def _mix(x):
    """32 well-mixed bits of each 32-bit number (held in int64)."""
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _dither(n, t):
    """16 random bits for m and for v of every entry at step t."""
    key = _mix(_mix(_mix(SEED & 0xFFFFFFFF) ^ (SEED >> 32)) ^ (t & 0xFFFFFFFF))
    h = _mix(torch.arange(n, device="cuda") ^ key)
    return (h & 0xFFFF).int(), (h >> 16).int()


def _encode(x, negative, top, bits, dither):
    """Codes and block scales of x (of |x| with the signs in `negative`)."""
    x = x.abs().view(-1, BLOCK)
    most = x.amax(1)
    held = (most >= TINY) & (most < math.inf)
    full = torch.full_like(most, top)
    inv = torch.where(held, full / most, torch.zeros_like(most))
    scale = torch.where(held, most / full, torch.where(most < TINY, torch.zeros_like(most), most * math.nan))
    y = x * inv[:, None] + 1.0
    k = y.view(torch.int32) + (dither.view(-1, BLOCK) << (7 - bits))
    k = ((k - (127 << 23)) >> (23 - bits)).clamp_(0, (16 << bits) - 1)
    if negative is None:      # the square root of a v that is not zero never becomes zero
        k = torch.where((k == 0) & (x > 0), torch.ones_like(k), k)
    k = torch.where(held[:, None], k, torch.zeros_like(k)).view(-1)
    if negative is not None:
        k = torch.where(negative, k + 128, k)
    return k.to(torch.uint8), scale


def _value(k, scale, bits):
    q = ((k.int() << (23 - bits)) + (127 << 23)).view(torch.float32) - 1.0
    return (q.view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_moments(s):
    mag = _value(s["m"] & 127, s["scales"][:, 0], M_BITS)
    r = _value(s["v"], s["scales"][:, 1], R_BITS)
    return torch.where(s["m"] >= 128, -mag, mag), r * r


def _plain_adamw(s):
    case, spans, s["t"] = s["case"], s["spans"], s["t"] + 1
    g = torch.zeros(s["n"], device="cuda")
    torch._foreach_copy_([g[a:b] for a, b in spans], s["grads"])
    if case["clip"]:
        norm = g.double().square_().sum().sqrt()
        g = g * torch.clamp(MAX_NORM / norm, max=1.0).float()
    m, v = (s["m"], s["v"]) if case["bits"] == 32 else _plain_moments(s)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + ((1 - BETA2) * g) * g
    if case["dtype"] == "bf16":
        p = s["master"]
    else:
        p = torch.zeros(s["n"], device="cuda")
        torch._foreach_copy_([p[a:b] for a, b in spans], s["params"])
    r = v.sqrt()
    step = LR * (math.sqrt(1.0 - BETA2 ** s["t"]) / (1.0 - BETA1 ** s["t"]))
    p = (p - step * (m / (r + ADAM_EPS))) * (1.0 - LR * DECAY)
    torch._foreach_copy_(s["params"], [p[a:b] for a, b in spans])
    out = {"params": s["param_flat"]}
    if case["dtype"] == "bf16":
        s["master"].copy_(p)
        out["master"] = s["master"]
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return out | {"m": s["m"], "v": s["v"]}
    for_m, for_v = _dither(s["n"], s["t"])
    s["m"], ms = _encode(m, m < 0, M_TOP, M_BITS, for_m)
    s["v"], vs = _encode(r, None, R_TOP, R_BITS, for_v)
    s["scales"] = torch.stack([ms, vs], 1)
    m, v = _plain_moments(s)
    return out | {"m": m, "v": v}


def _plain_ffn_fwd(s):
    x = s["x"].float()
    gate, up = x @ s["w_gate"].float(), x @ s["w_up"].float()
    h = _act(gate, s["case"]["act"]) * up
    out = {"h": h.bfloat16(), "y": (h @ s["w_down"].float()).bfloat16()}
    return out | {"gate": gate.bfloat16(), "up": up.bfloat16()} if s["case"]["train"] else out


def _plain_ffn_bwd(s):
    act, gate, up = s["case"]["act"], s["gate"].float(), s["up"].float()
    dy, x = s["dy"].float(), s["x"].float()
    dh = dy @ s["w_down"].float().t()
    dgate, dup = dh * up * _act_slope(gate, act), dh * _act(gate, act)
    return {"dx": (dgate @ s["w_gate"].float().t() + dup @ s["w_up"].float().t()).bfloat16(),
            "dw_gate": (x.t() @ dgate).bfloat16(), "dw_up": (x.t() @ dup).bfloat16(),
            "dw_down": (s["h"].float().t() @ dy).bfloat16()}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"adamw": _plain_adamw, "ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd}[op](s)
    import zero_sharded_adamw_gb300 as z
    stream = torch.cuda.current_stream()
    if op == "adamw":
        s["opt"].step(s["grad_table"], s["param_table"], s["master"], s["m"], s["v"], s["scales"], stream)
        out = {"params": s["param_flat"]}
        if s["master"] is not None:
            out["master"] = s["master"]
        if s["scales"] is None:
            return out | {"m": s["m"], "v": s["v"]}
        s["opt"].moments(s["m"], s["v"], s["scales"], s["m_out"], s["v_out"], stream)
        return out | {"m": s["m_out"], "v": s["v_out"]}
    if op == "ffn_fwd":
        train = s["case"]["train"]
        z.zero1_ffn_forward(s["shape"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"] if train else None,
                            s["up"] if train else None, s["h"], s["y"], s["workspace"], stream)
        out = {"h": s["h"], "y": s["y"]}
        return out | {"gate": s["gate"], "up": s["up"]} if train else out
    z.zero1_ffn_backward(s["shape"], s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"], s["h"],
                         s["dx"], s["dw_gate"], s["dw_up"], s["dw_down"], s["workspace"], stream)
    return {k: s[k] for k in ("dx", "dw_gate", "dw_up", "dw_down")}


# ------------------------------------------------------------------ work

def work(case):
    """Each input read once, each output written once.  An 8-bit state is read
    and written as codes and scales, and its values are written once."""
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        per = 2 + 2 + 8 if case["dtype"] == "bf16" else 4 + 8      # gradient, parameter, fp32 master
        per += 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8    # moments
        return {"bytes": per * n, "flops": 20 * n}
    rows, width, hidden = case["rows"], case["width"], case["hidden"]
    if case["op"] == "ffn_fwd":
        return {"bytes": 2 * (2 * rows * width + 3 * width * hidden + rows * hidden * (3 if case["train"] else 1)),
                "flops": 6 * rows * width * hidden}
    return {"bytes": 2 * (3 * rows * width + 6 * width * hidden + 3 * rows * hidden), "flops": 12 * rows * width * hidden}


# ----------------------------------------------------------------- exact

def _exact_adamw(s, case):
    """One step in 64 bits, tensor by tensor.  What 8 bits hold of the new
    moments goes by the random bits, so it has no exact value."""
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for grad in s["grads"]:
        total += torch.linalg.vector_norm(grad.double()) ** 2
    norm = float(total) ** 0.5
    coef = min(1.0, MAX_NORM / norm) if case["clip"] else 1.0
    t = STEPS_DONE + 1
    if case["bits"] == 32:
        m_all, v_all = s["m"].double(), s["v"].double()
    else:
        def grid(k, bits, scale):
            k = k.double()
            octave = torch.floor(k / 2 ** bits)
            value = torch.exp2(octave) * (1 + (k - octave * 2 ** bits) / 2 ** bits) - 1
            return value * scale.double().repeat_interleave(BLOCK)
        sign = 1.0 - 2.0 * (s["m"] > 127).double()
        m_all = sign * grid(s["m"].remainder(128), M_BITS, s["scales"][:, 0])
        v_all = grid(s["v"], R_BITS, s["scales"][:, 1]).square_()
    master = s["master"].double() if case["dtype"] == "bf16" else torch.zeros(s["n"], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(s["spans"]):
        p = master[a:b] if case["dtype"] == "bf16" else s["params"][i].double()
        g = s["grads"][i].double() * coef
        m = m_all[a:b].mul_(BETA1).add_(g, alpha=1 - BETA1)
        v = v_all[a:b].mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
        hat = (m / (1 - BETA1 ** t)) / (v.sqrt() + ADAM_EPS) * math.sqrt(1 - BETA2 ** t)
        master[a:b] = (p - LR * hat) * (1 - LR * DECAY)
    flat = torch.cat([master[a:b] for a, b in s["spans"]]) if case["packed"] else master
    out = {"params": flat, "m": m_all, "v": v_all} if case["bits"] == 32 else {"params": flat, "m": None, "v": None}
    return out | {"master": master} if case["dtype"] == "bf16" else out


def _gates64(g, act):
    """The activation and its derivative in 64 bits."""
    if act == "relu":
        return g.clamp(min=0), torch.heaviside(g, torch.zeros_like(g))
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * (1 - sig)
    if act == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    inner = torch.addcmul(c * g, g.square(), g, value=0.044715 * c)
    half = torch.sigmoid(2 * inner)                       # (1 + tanh(inner)) / 2
    return g * half, half + 2 * g * half * (1 - half) * (c + 3 * 0.044715 * c * g.square())


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s, case)
    x = s["x"].double()
    if case["op"] == "ffn_fwd":
        both = x @ torch.cat([s["w_gate"], s["w_up"]], 1).double()
        gate, up = both[:, :case["hidden"]], both[:, case["hidden"]:]
        h = _gates64(gate, case["act"])[0] * up
        out = {"h": h, "y": h @ s["w_down"].double()}
        return out | {"gate": gate.contiguous(), "up": up.contiguous()} if case["train"] else out
    dy = s["dy"].double()
    a, slope = _gates64(s["gate"].double(), case["act"])
    dh = torch.einsum("rw,hw->rh", dy, s["w_down"].double())
    both = torch.cat([dh * s["up"].double() * slope, dh * a], 1)
    weights = torch.cat([s["w_gate"], s["w_up"]], 1).double()
    dw = torch.einsum("rw,rh->wh", x, both)
    return {"dx": torch.einsum("rh,wh->rw", both, weights), "dw_gate": dw[:, :case["hidden"]].contiguous(),
            "dw_up": dw[:, case["hidden"]:].contiguous(), "dw_down": torch.einsum("rh,rw->hw", s["h"].double(), dy)}
