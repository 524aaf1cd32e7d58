"""The first call a process makes of the feed-forward block and of AdamW over a
list may be one that is being captured."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FFN = """
import torch
import tests.test_gpu_ffn as t
b = t.Block({rows}, 264, 520)
spaces = [b.space(k) for k in (False, True)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    cur = torch.cuda.current_stream()
    b.forward(stream=cur, space=spaces[0])
    b.backward(stream=cur, space=spaces[1])
graph.replay()
torch.cuda.synchronize()
b.check_forward()
b.check_backward()
"""

ADAMW = """
import torch
import tests.test_gpu_adamw_list as t
c = t.Case({sizes}, bits={bits})
c.draw()
want = c.plain()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    c.run(torch.cuda.current_stream())
graph.replay()
torch.cuda.synchronize()
c.check(want)
assert c.opt.steps() == 1
"""


@pytest.mark.parametrize("code", [FFN.format(rows=4), FFN.format(rows=100), FFN.format(rows=700),
                                  ADAMW.format(sizes=[300, 40], bits=8), ADAMW.format(sizes=[70000, 33], bits=8),
                                  ADAMW.format(sizes=[70000, 33], bits=32)],
                         ids=["few rows", "128 rows", "tiles", "one launch", "8 bits", "32 bits"])
def test_first_call_is_captured(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
