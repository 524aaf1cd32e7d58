"""Buffers that share memory in calls whose matrices have a single row (one
token; a width or hidden size of 1): refused wherever in the row the other
begins, without a GPU."""
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_ffn_cpu import bwd, fake, fwd


def passes(call, shape, **kw):
    """Neither the overlap nor the alignment of these buffers is refused: the check of the workspace comes next."""
    with pytest.raises(z.Zero1Error, match="workspace"):
        call(shape, **kw)


ROW = z.FfnShape(1, 4096, 16)           # x, y: one long row; h, gate, up: one short row
COLUMN = z.FfnShape(1, 768, 2048)       # h the longer
NARROW = z.FfnShape(40, 1, 4096)        # w_gate, w_up and their gradients: one row; w_down: one entry a row
THIN = z.FfnShape(40, 4096, 1)          # w_down and its gradient: one row


@pytest.mark.parametrize("call,shape,kw,word", [
    # inside the row, past the other's stride
    (fwd, ROW, dict(h=fake(0, 128)), "x and h share"),
    (fwd, ROW, dict(h=fake(0, 8176)), "x and h share"),
    (fwd, ROW, dict(gate=fake(0, 4096)), "x and gate share"),
    (fwd, ROW, dict(y=fake(0, 8176)), "x and y share"),
    (fwd, COLUMN, dict(y=fake(6, 1600)), "h and y share"),
    (fwd, COLUMN, dict(y=fake(6, 3200)), "h and y share"),
    (fwd, COLUMN, dict(w_down=fake(6, 4080)), "w_down and h share"),
    (fwd, COLUMN, dict(w_gate=fake(7, 1520)), "w_gate and y share"),
    # the row begins before, between and in the other's rows
    (fwd, ROW, dict(x=fake(6, -8160)), "x and h share"),
    (fwd, COLUMN, dict(y=fake(3, -1520)), "w_down and y share"),
    (fwd, COLUMN, dict(y=fake(3, 1536 * 100)), "w_down and y share"),
    (fwd, COLUMN, dict(h=fake(3, 1536 * 2047 + 1520)), "w_down and h share"),
    (bwd, ROW, dict(dx=fake(1, 8176)), "dx and x share"),
    (bwd, ROW, dict(dw_down=fake(0, 4096)), "dw_down and dy share"),
    (bwd, ROW, dict(dw_gate=fake(1, 8160)), "dw_gate and x share"),
    (bwd, NARROW, dict(dw_down=fake(2, 4096)), "dw_down and w_gate share"),
    (bwd, NARROW, dict(dw_gate=fake(4, 8176)), "dw_gate and w_down share"),
    (bwd, THIN, dict(dw_down=fake(2, 8176)), "dw_down and w_gate share"),
    (bwd, THIN, dict(dw_gate=fake(4, 8176)), "dw_gate and w_down share"),
])
def test_one_row_inside_another_buffer_is_refused(call, shape, kw, word):
    with pytest.raises(z.Zero1Error, match=word) as e:
        call(shape, **kw)
    assert e.value.code == -1


@pytest.mark.parametrize("call,shape,kw", [
    (fwd, ROW, dict(h=fake(0, 8192))), (fwd, ROW, dict(x=fake(6, -8192))),
    (fwd, COLUMN, dict(y=fake(6, 4096))), (fwd, COLUMN, dict(y=fake(6, -1536))),
    (fwd, COLUMN, dict(y=fake(3, 1536 * 2048))), (fwd, COLUMN, dict(h=fake(3, -4096))),
    (bwd, NARROW, dict(dw_down=fake(2, 8192))), (bwd, THIN, dict(dw_down=fake(2, -8192))),
    # a row between another's rows: its entries, not its extent, count
    (fwd, z.FfnShape(1, 16, 4096, ld_gate=8192), dict(h=fake(1, 8192))),
    (fwd, z.FfnShape(1, 16, 4096, ld_gate=8192), dict(h=fake(1, 8192 + 3 * 16384))),
])
def test_one_row_beside_another_buffer_is_taken(call, shape, kw):
    if torch.cuda.is_available() and z.zero1_ffn_workspace(shape, call is bwd) == 0:
        pytest.skip("the call would run")
    passes(call, shape, **kw)


def test_the_answer_is_that_of_the_entries():
    """Every place of a row against a small matrix, with and without gaps, compared with the sets of entries."""
    for rows, width, hidden, ld in ((1, 24, 8, 0), (1, 8, 24, 0), (1, 8, 16, 24), (1, 16, 8, 32)):
        shape = z.FfnShape(rows, width, hidden, ld_gate=ld, unaligned=True)
        stride = ld or hidden
        for offset in range(-2 * width - 4, 2 * (width * stride) + 4, 2):
            x = set(range(offset // 2, offset // 2 + width))
            w = {r * stride + c for r in range(width) for c in range(hidden)}
            kw = dict(y=fake(1, offset))
            if x & w:
                with pytest.raises(z.Zero1Error, match="w_gate and y share"):
                    fwd(shape, **kw)
            else:
                passes(fwd, shape, **kw)
