"""AdamW over a list that ends in a launch's worth of empty tensors, clipped."""
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_gpu_adamw_list import Case

pytestmark = pytest.mark.gpu


def steps_to_one(hp):
    """Entries of the bias corrections' table."""
    t = 1
    while hp.beta1 ** t > 2.0 ** -54 or hp.beta2 ** t > 2.0 ** -54:
        t += 1
    return t


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("empty", [1, 1600, 2000])
def test_the_norm_of_a_list_whose_last_tensors_are_empty(empty, bits):
    """1,600 tensors of 6,400 entries have as many partial sums as blocks that run at once; the launch behind them
    has no blocks of its own, but writes one more.  All of the handle's memory but these sums is known."""
    sizes = [6400] * 1600 + [0] * empty
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    hp = z.Hparams(max_norm=0.05)
    blocks = 1600 * 25
    sums = min(-(-blocks // 64), 4 * torch.cuda.get_device_properties(0).multi_processor_count) + 1
    with z.AdamW(sizes, hp, z.AdamWOptions(state_bits=bits)) as opt:
        held = opt.layout()[2] - 256 - up(4 * blocks) - up(8 * steps_to_one(hp))   # status, blocks, corrections
        assert held >= 8 * sums
    c = Case(sizes, bits=bits, hp=hp)
    for _ in range(2):
        c.draw()
        want = c.plain()
        c.run()
        c.check(want)
    assert c.opt.grad_norm()[1] == float(want["clip"]) < 1
