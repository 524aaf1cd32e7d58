"""The gated feed-forward block's activations where they are small, entry by
entry: a one-hot row of x picks one row of the weights, so gate and up are bf16
numbers that the test chooses and no sum stands between them and the result."""
import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import ffn_plain as fp
from tests.test_gpu_ffn import ACT, BF

pytestmark = pytest.mark.gpu


def run(rows, gates, name):
    """h of the forward pass, and dup and dgate of the backward one with dh = 1
    (as the weights' gradients of the row that x picks), each (hidden,)."""
    hidden, width = gates.numel(), 8
    wide = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    x, dy = wide(rows, width), wide(rows, width)
    x[:, 0] = 1.0
    dy[0, 0] = 1.0
    w_gate, w_up, w_down = wide(width, hidden), wide(width, hidden), wide(hidden, width)
    w_gate[0], w_up[0], w_down[:, 0] = gates, 1.0, 1.0
    gate, up, h = wide(rows, hidden), wide(rows, hidden), wide(rows, hidden)
    y, dx, dwg, dwu, dwd = wide(rows, width), wide(rows, width), wide(width, hidden), wide(width, hidden), wide(hidden, width)
    s = z.FfnShape(rows, width, hidden, ACT[name])
    space = torch.empty(max(z.zero1_ffn_workspace(s, k) for k in (False, True)), dtype=torch.uint8, device="cuda")
    z.zero1_ffn_forward(s, x, w_gate, w_up, w_down, gate, up, h, y, space)
    z.zero1_ffn_backward(s, dy, x, w_gate, w_up, w_down, gate, up, h, dx, dwg, dwu, dwd, space)
    assert torch.equal(gate, gates.expand(rows, hidden)) and bool((up == 1).all()) and torch.equal(h, h[:1].expand_as(h))
    return h[0], dwu[0], dwg[0]


def exact(g, name):
    """The activation and its derivative in 64 bits; the tanh form by (1 + tanh z)/2 = sigmoid(2 z), which does not cancel."""
    if name != "gelu_tanh":
        return fp.act(g, name)
    k = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))
    return g * s, s + 2 * g * s * torch.sigmoid(-2 * k * (g + 0.044715 * g ** 3)) * k * (1 + 3 * 0.044715 * g * g)


def check(rows, gates, name, slack):
    """Each value is rounded to bf16 once (dup and dgate twice, the second time
    exactly: E), after an activation that is `slack` off relatively."""
    a, slope = exact(gates.double(), name)
    for got, want, what in zip(run(rows, gates, name), (a, a, slope), ("h", "dup", "dgate")):
        off = want.abs() * (fp.E + slack) + 1e-37
        bad = ~((got.double() - want).abs() <= off)
        assert not bool(bad.any()), (what, gates[bad].tolist()[:4], got[bad].tolist()[:4], want[bad].tolist()[:4])


# Rows: few, at most 128, and tiles.
@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("name", fp.ACTS)
def test_tails_keep_their_relative_accuracy(rows, name):
    """Every bf16 gate from -8 to -2 and from 2 to 8.  The activations' functions in fp32, relative to themselves:
    exp of at most 49 in magnitude 2 + 1.17 * 49 = 60 units of 2^-23, and its argument's six roundings times 49:
    2.5e-5 (that of g^2/2 = 32 at most: 1e-5, with the fitted quotient's 6e-7); the slopes' two terms cancel to no
    less than 0.27 of their sum of magnitudes (SiLU at -2): 2.5e-5 / 0.27 = 9.3e-5, and products: 1e-4."""
    gates = torch.arange(0x4000, 0x4101, dtype=torch.int32, device="cuda").to(torch.int16).view(BF)
    check(rows, torch.cat([gates, -gates])[:512], name, 1e-4)


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("name", fp.ACTS)
def test_gates_up_to_the_largest(rows, name):
    """Where g^2 and g^3 leave fp32's range the activation is g or 0 and its slope 1 or 0."""
    big = [1e2, 1e5, 1e10, 1e13, 1e15, 1e18, 2e19, 1e20, 1e30, 3e38]
    gates = torch.tensor([s * v for v in big for s in (1, -1)], device="cuda").to(BF)
    check(rows, torch.cat([gates, gates.new_ones(4)]), name, 1e-4)
