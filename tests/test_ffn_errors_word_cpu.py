"""The feed-forward block's error word inside a matrix or the workspace is
refused, and between a matrix's rows it is not; without a GPU."""
import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_ffn_cpu import bwd, fake, fwd

SHAPE = z.FfnShape(40, 16, 32)
GAPS = z.FfnShape(40, 16, 32, ldy=24, ldh=48)


@pytest.mark.parametrize("call,at,word", [
    (fwd, fake(0), "errors and x share"), (fwd, fake(0, 40 * 32 - 4), "errors and x share"),
    (fwd, fake(3, 64), "errors and w_down share"), (fwd, fake(6, 1280), "errors and h share"), (fwd, fake(7, 4), "errors and y share"),
    (bwd, fake(0, 32), "errors and dy share"), (bwd, fake(8), "errors and dx share"), (bwd, fake(11, 1020), "errors and dw_down share"),
    (bwd, fake(5, 2556), "errors and gate share"),
])
def test_inside_a_matrix(call, at, word):
    with pytest.raises(z.Zero1Error, match=word) as e:
        call(SHAPE, errors=at)
    assert e.value.code == -1


@pytest.mark.parametrize("call,shape,at", [
    (bwd, SHAPE, fake(0, 40 * 32)), (bwd, SHAPE, fake(0, -4)),
    (bwd, GAPS, fake(0, 32)), (bwd, GAPS, fake(0, 44)), (bwd, GAPS, fake(5, 5 * 96 + 64)),
])
def test_beside_a_matrix_or_between_its_rows(call, shape, at):
    with pytest.raises(z.Zero1Error, match="workspace holds 0 bytes"):
        call(shape, errors=at)


def test_between_rows_but_reaching_into_one():
    with pytest.raises(z.Zero1Error, match="errors and dy share"):
        bwd(z.FfnShape(40, 16, 32, ldy=17, unaligned=True), errors=fake(0, 32))


@pytest.mark.parametrize("inside", [0, 252])
def test_inside_the_workspace(inside):
    need = z.zero1_ffn_workspace(SHAPE, True)

    class Space:
        is_cuda, nbytes = True, need + 4096

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return fake(20)

    with pytest.raises(z.Zero1Error, match="errors lies in the workspace"):
        bwd(SHAPE, workspace=Space(), errors=fake(20, inside))
    if not torch.cuda.is_available():
        with pytest.raises(z.Zero1Error, match="device query|no CUDA|driver|ECUDA"):    # what the call does not use is free
            bwd(SHAPE, workspace=Space(), errors=fake(20, need))


def test_a_host_tensor_is_no_error_word():
    for call in (fwd, bwd):
        with pytest.raises(z.Zero1ArgumentError, match="errors: expected a CUDA tensor"):
            call(SHAPE, errors=torch.zeros(1, dtype=torch.int32))


def test_a_tensor_smaller_than_the_word():
    class Word:
        is_cuda, nbytes = True, 2

        def data_ptr(self):
            return fake(20)

    with pytest.raises(z.Zero1ArgumentError, match="errors: 2 bytes"):
        fwd(SHAPE, errors=Word())
