"""What a list handle's binding keeps of the options it was created with,
against a stand-in for the library (creation needs a device)."""
import pytest

import zero_sharded_adamw_gb300 as z


class Library:
    """Accepts every call and records the steps'."""

    def __init__(self):
        self.made, self.steps = 0, []

    def zero1_adamw_create(self, sizes, decays, count, hp, opts, out):
        self.made += 1
        out._obj.value = 0x1000 + self.made
        return 0

    def zero1_adamw_step(self, h, grads, params, master, m, v, scales, stream):
        self.steps.append((h, m, v))
        return 0

    def zero1_adamw_layout(self, h, entries, starts, device_bytes):
        entries._obj.value = 256
        return 0

    def zero1_adamw_destroy(self, h):
        return 0

    def zero1_last_error(self):
        return b""


class Tensor:
    """A CUDA tensor, as far as the checks look."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, dtype, count):
        self.dtype, self.count = dtype, count

    def numel(self):
        return self.count

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


BF, F32, U8 = "torch.bfloat16", "torch.float32", "torch.uint8"


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(z, "_lib", lib)
    for table in ("_ADAMW_HANDLES", "_DTYPE_NAMES", "_TORCH_DTYPES"):
        monkeypatch.setattr(z, table, {})
    return lib


def step(opt, moments, grad=BF, param=BF, scales=None):
    opt.step([Tensor(grad, 200)], [Tensor(param, 200)], Tensor(F32, 256) if param == BF else None, Tensor(moments, 256),
             Tensor(moments, 256), scales)


def test_options_changed_after_creation_do_not_reach_the_handle(lib):
    opts = z.AdamWOptions()
    first = z.AdamW([200], opts=opts)
    opts.state_bits = 8
    second = z.AdamW([200], opts=opts)
    opts.param_dtype = opts.grad_dtype = z.DTYPE_F32
    third = z.AdamW([200], opts=opts)
    opts.state_bits, opts.seed = 32, 9
    # each is stepped with the buffers it was created for
    step(first, F32)
    step(second, U8, scales=Tensor(F32, 2))
    step(third, U8, F32, F32, scales=Tensor(F32, 2))
    assert [s[0] for s in lib.steps] == [first.handle, second.handle, third.handle]
    # and bytes are never taken for a handle of fp32 moments, nor fp32 for bytes
    for opt, moments, grad, word in ((first, U8, BF, "m: expected torch.float32"), (second, F32, BF, "m: expected torch.uint8"),
                                     (first, F32, F32, "grads\\[0\\]: expected torch.bfloat16"),
                                     (third, U8, BF, "grads\\[0\\]: expected torch.float32")):
        with pytest.raises(z.Zero1ArgumentError, match=word):
            step(opt, moments, grad, grad)
    assert len(lib.steps) == 3
    assert (first.opts.state_bits, second.opts.state_bits, third.opts.grad_dtype) == (32, 8, z.DTYPE_F32)
    assert (first.scale_entries, second.scale_entries) == (0, 2)


def test_the_wrappers_own_options_are_no_way_in(lib):
    opt = z.AdamW([200])
    opt.opts.state_bits = 8
    step(opt, F32)
    with pytest.raises(z.Zero1ArgumentError, match="m: expected torch.float32"):
        step(opt, U8)


def test_hyperparameters_are_those_of_creation(lib):
    hp = z.Hparams(lr=1e-3)
    opt = z.AdamW([200], hp)
    hp.lr = 5.0
    assert opt.hp.lr == 1e-3
