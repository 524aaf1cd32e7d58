"""How far 8-bit moments let v come out high: rounding at random keeps the mean
of sqrt(v), so v gains the rounding's variance."""
import math

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests import adamw_plain as ap
from tests.test_gpu_adamw_list import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beta2,steps", [(0.95, 40), (0.999, 1000)])
def test_v_gains_the_variance_of_its_roots_rounding(beta2, steps):
    """In every block one entry's gradient holds the largest v, and with it the block's scale, at 1; the others'
    gradients are zero, and their roots fall by a fraction d = 1 - sqrt(beta2) a step, less than the gap to the code
    below, a fraction w of them.  A root that was a code becomes that or the one below, with variance d (w - d) of
    its square, so a step multiplies v's mean by beta2 + d (w - d).  w is 1/32 (from an octave's first code) to
    1/17 (its second), times value + 1 over value: 1.0005 at the octaves looked at.  The spread of an entry's
    root after all steps is sqrt(steps d w) = 0.25 at most, of v twice that, of the mean of 65,280 entries 0.2%;
    six times that is allowed."""
    hp = z.Hparams(beta2=beta2, lr=0.0, max_norm=0.0)
    c = Case([65536], "f32", "f32", 8, hp=hp)
    largest = torch.arange(0, 65536, 256, device="cuda")
    c.v.copy_(torch.randint(200, 255, (65536,), generator=c.gen, device="cuda"))
    c.v[largest] = 255
    c.scales.view(-1, 2)[:, 1] = 1.0 / ap.R_TOP
    c.grads[0].zero_()
    c.grads[0][largest] = 1.0
    others = torch.ones(65536, dtype=torch.bool, device="cuda")
    others[largest] = False
    before = float(c.moments()[1][others].double().sum())
    for _ in range(steps):
        c.run()
    v = c.moments()[1].double()
    assert float((v[largest].sqrt() - 1).abs().max()) <= 1 / 16     # the scale stayed (but for a code, now and then)
    gain = float(v[others].sum()) / before / beta2 ** steps
    d = 1 - math.sqrt(beta2)
    low, high = ((1 + d * (w - d) / beta2) ** steps for w in (1 / 32, 1.0005 / 17))
    spread = 6 * 2 * math.sqrt(steps * d * 1.0005 / 17 / 65280)
    assert low - spread <= gain <= high + spread, (low, gain, high)
