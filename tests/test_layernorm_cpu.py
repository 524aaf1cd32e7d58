"""Layer norm's argument checks, which come before any device call, and its
workspace size."""
from __future__ import annotations

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from zero_sharded_adamw_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def forward(rows=4, cols=8, dtype=z.DTYPE_F32, x=16, ldx=8, gamma=16, beta=16, eps=1e-5, y=16, ldy=8, mean=16, rstd=16):
    z.zero1_layernorm_forward(rows, cols, dtype, x, ldx, gamma, beta, eps, y, ldy, mean, rstd)


@pytest.mark.parametrize("kw,code", [
    (dict(cols=0), -1), (dict(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25), -1), (dict(rows=1 << 31), -1),
    (dict(dtype=2), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(ldx=7), -1), (dict(ldy=7), -1),
    (dict(x=None), -1), (dict(gamma=None), -1), (dict(y=None), -1), (dict(mean=None), -1), (dict(rstd=None), -1),
    (dict(x=18), -2), (dict(gamma=17), -2), (dict(beta=18), -2), (dict(y=2), -2), (dict(mean=2), -2), (dict(rstd=2), -2),
    (dict(dtype=z.DTYPE_BF16, x=17), -2),
])
def test_forward_refusals(kw, code):
    with pytest.raises(z.Zero1Error) as e:
        forward(**kw)
    assert e.value.code == code


def test_no_rows_is_no_work():
    forward(rows=0, x=None, gamma=None, y=None, mean=None, rstd=None)


def test_workspace():
    assert z.zero1_layernorm_workspace(0, 5) == 2 * 5 * 4
    assert z.zero1_layernorm_workspace(7, 5) == 7 * 2 * 5 * 4
    assert z.zero1_layernorm_workspace(10**6, 768) == 320 * 2 * 768 * 4
    for rows, cols in ((1, 0), (1 << 31, 8), (1, (1 << 24) + 1)):
        with pytest.raises(z.Zero1Error) as e:
            z.zero1_layernorm_workspace(rows, cols)
        assert e.value.code == -1


def backward(workspace_bytes=4 * 2 * 8 * 4, **kw):
    a = dict(rows=4, cols=8, dtype=z.DTYPE_F32, dy=16, lddy=8, x=16, ldx=8, gamma=16, mean=16, rstd=16, dx=16, lddx=8,
             dgamma=16, dbeta=16, grad_dtype=z.DTYPE_F32, workspace=16)
    a.update(kw)
    z._check(z._load().zero1_layernorm_backward(*list(a.values()), workspace_bytes, None))


@pytest.mark.parametrize("kw,code", [
    (dict(cols=0), -1), (dict(dtype=5), -1), (dict(grad_dtype=5), -1), (dict(lddy=7), -1), (dict(ldx=7), -1),
    (dict(lddx=7), -1), (dict(dy=None), -1), (dict(x=None), -1), (dict(gamma=None), -1), (dict(mean=None), -1),
    (dict(rstd=None), -1), (dict(dx=None), -1), (dict(dgamma=None), -1), (dict(workspace=None), -1),
    (dict(workspace_bytes=4 * 2 * 8 * 4 - 1), -1), (dict(workspace=8), -2), (dict(dy=18), -2), (dict(dgamma=18), -2),
    (dict(dbeta=17, grad_dtype=z.DTYPE_BF16), -2), (dict(dx=2), -2),
])
def test_backward_refusals(kw, code):
    with pytest.raises(z.Zero1Error) as e:
        backward(**kw)
    assert e.value.code == code


def test_binding_checks_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(z.Zero1ArgumentError, match="CUDA"):
        forward(x=x)
    with pytest.raises(z.Zero1ArgumentError, match="bfloat16"):
        forward(dtype=z.DTYPE_BF16, x=x)
    with pytest.raises(z.Zero1ArgumentError, match="workspace"):
        z.zero1_layernorm_backward(4, 8, z.DTYPE_F32, 16, 8, 16, 8, 16, 16, 16, 16, 8, 16, 16, z.DTYPE_F32, 16)


@pytest.mark.parametrize("ld", [-1, 1 << 63, (1 << 49) + 1])
def test_strides_past_any_memory_are_refused(ld):
    for call, names in ((forward, ("ldx", "ldy")), (backward, ("lddy", "ldx", "lddx"))):
        for name in names:
            with pytest.raises(z.Zero1Error) as e:
                call(**{name: ld})
            assert e.value.code == -1, name


def test_in_place_needs_one_stride():
    for call, kw in ((forward, dict(ldy=16)), (backward, dict(lddx=16))):
        with pytest.raises(z.Zero1Error) as e:
            call(**kw)
        assert e.value.code == -1 and "same row stride" in str(e.value)


class FakeCuda:
    """A CPU tensor that says it is on the device; only its shape is looked at."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_refuses_rows_with_gaps():
    for x in (torch.zeros(64)[::2], torch.zeros(4, 16)[:, ::2], torch.zeros(8, 4).t()):
        with pytest.raises(z.Zero1ArgumentError, match="adjacent"):
            z._take_rows(FakeCuda(x), 4, 8, 8, "f32", "x")
    for x in (torch.zeros(32), torch.zeros(4, 8), torch.zeros(1, 32)):
        assert z._take_rows(FakeCuda(x), 4, 8, 8, "f32", "x") == x.data_ptr()
