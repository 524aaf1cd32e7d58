"""AdamW over a list: tensors inside the state are refused before anything runs."""
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_gpu_adamw_list import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", ["bf16", "f32"])
def test_tensors_inside_the_state_are_refused(bits, param):
    c = Case([300, 40], param, "f32", bits)
    c.draw()
    want = c.plain()
    before = [x.clone() for x in c.params]
    f32 = lambda x, n: x.view(torch.float32)[:n]  # noqa: E731
    buffers = {"m": c.m, "v": c.v} | ({"master": c.master} if param == "bf16" else {}) | ({"scales": c.scales} if bits == 8 else {})
    for name, x in buffers.items():
        inside = f32(x, min(40, x.view(torch.float32).numel())) if name != "scales" else x
        grads, params = list(c.grads), list(c.params)
        at = inside.data_ptr()
        for lists, kind in ((dict(grads=[grads[0], at]), "gradient"), (dict(params=[params[0], at]), "parameter")):
            with pytest.raises(z.Zero1Error, match=f"the {kind} of tensor 1 shares memory with {name}"):
                c.opt.step(**{**dict(grads=grads, params=params, master=c.master, m=c.m, v=c.v, scales=c.scales), **lists})
    assert c.opt.steps() == 0 and all(torch.equal(a, b) for a, b in zip(before, c.params))
    c.run()
    c.check(want)
