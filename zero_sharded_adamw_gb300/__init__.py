"""GB300 (sm_103a) ZeRO-1 data-parallel optimizer step.

A thin ctypes binding of ``libzero1.so`` (C ABI in ``include/zero1.h``): the
functions below carry the C entry points' names and only marshal arguments.
Every step of the path runs in the library's CUDA kernels; there is no
CPU fallback.  The library is built by ``__graft_entry__.build()`` (or
``python -m zero_sharded_adamw_gb300._build``); calling any entry point
without it raises ``Zero1Error``.

Pointers may be given as ints or as objects with ``data_ptr()`` (torch
tensors) or ``ctypes.data`` (numpy arrays).  Streams may be ints, objects
with ``cuda_stream`` (torch streams) or None (the legacy default stream).
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, replace

__all__ = [
    "Zero1Error", "Zero1ArgumentError", "Hparams", "Options", "Zero1", "PtrTable",
    "zero1_create", "zero1_create_ex", "zero1_destroy", "zero1_step", "zero1_step_host",
    "zero1_step_host_async", "zero1_host_sync",
    "zero1_set_state", "zero1_get_state", "zero1_set_state_range", "zero1_get_state_range",
    "zero1_set_lr", "zero1_set_lr_ptr", "zero1_get_grad_norm",
    "zero1_layout", "zero1_bucket_begin", "zero1_bucket_reduce", "zero1_bucket_update", "zero1_bucket_finish", "zero1_profile_start", "zero1_profile_stop", "zero1_profile_read", "zero1_step_launches", "zero1_shard_plan", "zero1_step_scalars", "zero1_step_noalloc", "zero1_allreduce", "zero1_allreduce_sum", "zero1_allgather", "zero1_last_error",
    "SmPartition", "zero1_sm_partition_create", "zero1_sm_partition_destroy",
    "MuonHparams", "Muon", "zero1_muon_create", "zero1_muon_destroy", "zero1_muon_step", "zero1_muon_orthogonalize",
    "zero1_muon_set_lr", "zero1_muon_status", "zero1_muon_layout",
    "zero1_layernorm_forward", "zero1_layernorm_backward", "zero1_layernorm_workspace",
    "ACT_SILU", "ACT_GELU", "ACT_GELU_TANH", "ACT_RELU", "FfnShape", "zero1_ffn_workspace", "zero1_ffn_forward",
    "zero1_ffn_backward",
    "AdamWOptions", "AdamW", "zero1_adamw_create", "zero1_adamw_destroy", "zero1_adamw_step", "zero1_adamw_moments",
    "zero1_adamw_set_steps", "zero1_adamw_set_lr", "zero1_adamw_get_steps", "zero1_adamw_get_grad_norm",
    "zero1_adamw_layout",
    "library_path", "EXPORTED_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libzero1.so")

ZERO1_MAX_WORLD = 512
ERRORS = {-1: "ZERO1_EINVAL", -2: "ZERO1_EALIGN", -3: "ZERO1_ENOMEM", -4: "ZERO1_ECUDA", -5: "ZERO1_ENODEV"}

# Every entry point include/zero1.h declares, with its ctypes signature.
_P, _U64, _I32, _F64 = C.c_void_p, C.c_uint64, C.c_int, C.c_double
_SIGS = {
    "zero1_create": (_I32, [_U64, _I32, _P, _P]),
    "zero1_create_ex": (_I32, [_U64, _I32, _P, _P, _P]),
    "zero1_destroy": (_I32, [_P]),
    "zero1_step": (_I32, [_P, _P, _P, _P]),
    "zero1_step_host": (_I32, [_P, _P, _P, _P]),
    "zero1_step_host_async": (_I32, [_P, _P, _P, _P]),
    "zero1_host_sync": (_I32, [_P]),
    "zero1_set_state": (_I32, [_P, _P, _P, _P, _U64, _P]),
    "zero1_get_state": (_I32, [_P, _P, _P, _P, _P, _P]),
    "zero1_set_state_range": (_I32, [_P, _U64, _U64, _P, _P, _P, _P]),
    "zero1_get_state_range": (_I32, [_P, _U64, _U64, _P, _P, _P, _P]),
    "zero1_set_lr": (_I32, [_P, _F64]),
    "zero1_set_lr_ptr": (_I32, [_P, _P]),
    "zero1_get_grad_norm": (_I32, [_P, _P, _P, _P]),
    "zero1_layout": (_I32, [_P, _P, _P, _P]),
    "zero1_bucket_begin": (_I32, [_P]),
    "zero1_bucket_reduce": (_I32, [_P, _U64, _U64, _P, _P]),
    "zero1_bucket_update": (_I32, [_P, _U64, _U64, _P, _P, _P]),
    "zero1_bucket_finish": (_I32, [_P, _P, _P]),
    "zero1_profile_start": (_I32, [_P, _I32]),
    "zero1_profile_stop": (_I32, [_P, _P, _P, _P]),
    "zero1_profile_read": (_I32, [_P, _P, _P, _U64, _P]),
    "zero1_step_launches": (_I32, [_P, _P]),
    "zero1_shard_plan": (_I32, [_U64, _I32, _P, _P]),
    "zero1_step_scalars": (_I32, [_P, _I32, _U64, _P]),
    "zero1_step_noalloc": (_I32, [_U64, _I32, _P, _U64, _P, _P, _P, _P, _P, _P]),
    "zero1_allreduce": (_I32, [_U64, _I32, _I32, _I32, _P, _P, _P, _P]),
    "zero1_allreduce_sum": (_I32, [_P, _P, _P, _P]),
    "zero1_allgather": (_I32, [_U64, _I32, _U64, _I32, _P, _P, _P, _P]),
    "zero1_sm_partition_create": (_I32, [_I32, _P]),
    "zero1_sm_partition_destroy": (_I32, [_P]),
    "zero1_muon_create": (_I32, [_U64, _I32, _P, _U64, _P, _P]),
    "zero1_muon_destroy": (_I32, [_P]),
    "zero1_muon_step": (_I32, [_P, _P, _P, _P, _P, _P]),
    "zero1_muon_orthogonalize": (_I32, [_P, _P, _I32, _P, _I32, _P]),
    "zero1_muon_set_lr": (_I32, [_P, _F64]),
    "zero1_muon_status": (_I32, [_P, _P]),
    "zero1_muon_layout": (_I32, [_P, _P, _P]),
    "zero1_layernorm_forward": (_I32, [_U64, _U64, _I32, _P, _U64, _P, _P, _F64, _P, _U64, _P, _P, _P]),
    "zero1_layernorm_workspace": (_I32, [_U64, _U64, _P]),
    "zero1_layernorm_backward": (_I32, [_U64, _U64, _I32, _P, _U64, _P, _U64, _P, _P, _P, _P, _U64, _P, _P, _I32, _P,
                                        _U64, _P]),
    "zero1_ffn_workspace": (_I32, [_P, _I32, _P]),
    "zero1_ffn_forward": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _U64, _P, _P]),
    "zero1_ffn_backward": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _U64, _P, _P]),
    "zero1_adamw_create": (_I32, [_P, _P, _U64, _P, _P, _P]),
    "zero1_adamw_destroy": (_I32, [_P]),
    "zero1_adamw_step": (_I32, [_P, _P, _P, _P, _P, _P, _P, _P]),
    "zero1_adamw_moments": (_I32, [_P, _P, _P, _P, _P, _P, _P]),
    "zero1_adamw_set_steps": (_I32, [_P, _U64, _P]),
    "zero1_adamw_set_lr": (_I32, [_P, _F64, _P]),
    "zero1_adamw_get_steps": (_I32, [_P, _P, _P]),
    "zero1_adamw_get_grad_norm": (_I32, [_P, _P, _P, _P]),
    "zero1_adamw_layout": (_I32, [_P, _P, _P, _P]),
    "zero1_last_error": (C.c_char_p, []),
}
EXPORTED_SYMBOLS = tuple(_SIGS)


class Zero1Error(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{ERRORS.get(code, code)}: {message}")
        self.code = code


class Zero1ArgumentError(Zero1Error, ValueError):
    """An argument the binding refused before calling the library (a pointer
    list whose length is not the world size, a buffer of the wrong type,
    place or size): code ZERO1_EINVAL, like the library's own checks."""

    def __init__(self, message: str):
        super().__init__(-1, message)


class _CHparams(C.Structure):
    _fields_ = [(k, C.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay", "max_norm")]


@dataclass
class Hparams:
    """AdamW + clipping hyperparameters; max_norm <= 0 disables clipping."""
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.95
    eps: float = 1e-8
    weight_decay: float = 0.1
    max_norm: float = 1.0

    def _c(self) -> _CHparams:
        return _CHparams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, self.max_norm)


class _COptions(C.Structure):
    _fields_ = [("size", C.c_uint32), ("decay_before_update", C.c_int32), ("clip_eps", C.c_double),
                ("moments_bf16", C.c_int32), ("bucket_ctas", C.c_int32), ("small_step", C.c_int32),
                ("capturable", C.c_int32), ("inject_wait_timeout", C.c_int32), ("host_chunk", C.c_uint64),
                ("load_phase_gbs", C.c_double)]


@dataclass
class Options:
    """Step variants: torch.optim.AdamW's decay order, a clip eps (torch's
    clip_grad_norm_ uses 1e-6), m and v stored in bf16; the bucketed step's
    CTAs per bucket; the one-launch small-n path (0 auto, 1 on, -1 off);
    capturable steps (device-side step counter and lr, for CUDA graphs);
    the host-buffer steps' chunk size; the update kernel's load phasing
    (0 = built-in rule, > 0 = device-wide rate in GB/s, < 0 = off)."""
    decay_before_update: bool = False
    clip_eps: float = 0.0
    moments_bf16: bool = False
    bucket_ctas: int = 0
    small_step: int = 0
    capturable: bool = False
    inject_wait_timeout: bool = False    # failure testing: the update kernel's waits run out
    host_chunk: int = 0                  # host-buffer steps: parameters per chunk (0 = default)
    load_phase_gbs: float = 0.0          # update-kernel load phasing: 0 built-in, > 0 rate (GB/s), < 0 off

    def _c(self) -> _COptions:
        return _COptions(C.sizeof(_COptions), 1 if self.decay_before_update else 0, self.clip_eps,
                         1 if self.moments_bf16 else 0, self.bucket_ctas, self.small_step,
                         1 if self.capturable else 0, 1 if self.inject_wait_timeout else 0, self.host_chunk,
                         self.load_phase_gbs)


_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise Zero1Error(-5, f"{_LIB_PATH} is not built; run "
                                 "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != 0:
        raise Zero1Error(rc, _load().zero1_last_error().decode())


def _addr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    if hasattr(x, "ctypes"):
        return int(x.ctypes.data)
    raise TypeError(f"cannot take the address of {type(x).__name__}")


def _stream(s) -> int | None:
    if s is None:
        return None
    if isinstance(s, int):
        return s or None
    return int(s.cuda_stream) or None


class PtrTable:
    """A pointer array built once (W buffers' addresses), for callers that
    pass the same buffers every step: it skips the per-call marshalling.
    It keeps references to the buffers so that they outlive the table."""

    def __init__(self, xs):
        self.buffers = list(xs)
        self.array = (C.c_void_p * len(self.buffers))(*[_addr(x) for x in self.buffers])
        self._checked: set = set()       # (count, kind, on_device) already validated

    def __len__(self) -> int:
        return len(self.buffers)


# Element kinds a C entry point expects behind a pointer: torch dtype name
# and element size in bytes.
_KINDS = {"bf16": ("torch.bfloat16", 2), "f32": ("torch.float32", 4), "u8": ("torch.uint8", 1)}
_DTYPE_NAMES: dict = {}    # torch dtype -> its name (naming one takes longer than the other checks together)
_TORCH_DTYPES: dict = {}   # element kind -> torch dtype, as they are met


def _dtype_name(x) -> str:
    d = x.dtype
    name = _DTYPE_NAMES.get(d)
    if name is None:
        name = _DTYPE_NAMES[d] = str(d)
        _TORCH_DTYPES.update({kind: d for kind, (want, _) in _KINDS.items() if want == name})
    return name


def _take(x, count: int, kind: str, what: str, rank: int | None = None) -> int | None:
    """Address of device buffer `x` (of that rank) after _check_buffer, whose
    tests an ordinary CUDA tensor passes here in one line."""
    try:
        if x.dtype is _TORCH_DTYPES[kind] and x.is_cuda and x.is_contiguous() and x.numel() >= count:
            return x.data_ptr()
    except (AttributeError, KeyError):
        pass
    _check_buffer(x, count, kind, True, what if rank is None else f"{what}[{rank}]")
    return _addr(x)


def _check_buffer(x, count: int, kind: str, on_device: bool | None, what: str) -> None:
    """Raise ValueError unless buffer `x` can hold `count` elements of `kind`
    where the C side will look for them (on_device: True = CUDA memory,
    False = host memory, None = either).  Raw integer addresses and None
    pass unchecked: only objects that describe themselves can be checked."""
    if x is None or isinstance(x, int):
        return
    want, size = _KINDS[kind]
    if hasattr(x, "data_ptr") and hasattr(x, "numel"):          # torch tensor
        if _dtype_name(x) != want:
            raise Zero1ArgumentError(f"{what}: expected {want}, got {x.dtype}")
        if on_device is not None and bool(x.is_cuda) != on_device:
            raise Zero1ArgumentError(f"{what}: expected a {'CUDA' if on_device else 'host'} tensor, got {x.device}")
        if not x.is_contiguous():
            raise Zero1ArgumentError(f"{what}: tensor is not contiguous")
        if x.numel() < count:
            raise Zero1ArgumentError(f"{what}: {x.numel()} elements, the call reads or writes {count}")
    elif hasattr(x, "ctypes") and hasattr(x, "nbytes"):          # numpy array (host memory)
        if on_device:
            raise Zero1ArgumentError(f"{what}: a numpy array is host memory; this argument must be device memory")
        if x.itemsize != size:
            raise Zero1ArgumentError(f"{what}: {x.itemsize}-byte elements, expected {size}-byte {kind}")
        if not x.flags["C_CONTIGUOUS"]:
            raise Zero1ArgumentError(f"{what}: array is not contiguous")
        if x.size < count:
            raise Zero1ArgumentError(f"{what}: {x.size} elements, the call reads or writes {count}")


def _ptrs(xs, world: int | None = None, count: int | None = None, kind: str | None = None,
          on_device: bool | None = True, what: str = "buffers") -> C.Array:
    """The host array of W pointers the C side reads.  With `world` it must
    hold exactly W entries (the C side reads W of them); with `count` and
    `kind` every buffer is checked to hold that many elements of that type."""
    n = len(xs)
    if world is not None and n != world:
        raise Zero1ArgumentError(f"{what}: {n} pointers given, the call reads {world}")
    if isinstance(xs, PtrTable):
        if count is not None and kind is not None:
            key = (count, kind, on_device)
            if key not in xs._checked:
                for r, x in enumerate(xs.buffers):
                    _check_buffer(x, count, kind, on_device, f"{what}[{r}]")
                xs._checked.add(key)
        return xs.array
    if count is not None and kind is not None:
        if on_device:
            return (C.c_void_p * n)(*[_take(x, count, kind, what, r) for r, x in enumerate(xs)])
        for r, x in enumerate(xs):
            _check_buffer(x, count, kind, on_device, f"{what}[{r}]")
    return (C.c_void_p * n)(*[_addr(x) for x in xs])


# (n, world, moments in bf16) of every handle this binding created, so that
# the per-call checks know the sizes the C side will use.
_HANDLES: dict[int, tuple[int, int, bool]] = {}


def _info(h) -> tuple[int | None, int | None, bool]:
    return _HANDLES.get(h, (None, None, False))


# --------------------------------------------------------- entry points

def zero1_last_error() -> str:
    return _load().zero1_last_error().decode()


def zero1_create(n: int, world: int, hp: Hparams | None = None) -> int:
    """Create a handle for n parameters over `world` emulated ranks."""
    h = C.c_void_p()
    c = (hp or Hparams())._c()
    _check(_load().zero1_create(n, world, C.byref(c), C.byref(h)))
    _HANDLES[h.value] = (n, world, False)
    return h.value


def zero1_create_ex(n: int, world: int, hp: Hparams | None = None, opts: Options | None = None) -> int:
    """Create a handle with step variants."""
    h = C.c_void_p()
    c = (hp or Hparams())._c()
    o = (opts or Options())._c()
    _check(_load().zero1_create_ex(n, world, C.byref(c), C.byref(o), C.byref(h)))
    _HANDLES[h.value] = (n, world, bool(opts and opts.moments_bf16))
    return h.value


def zero1_destroy(h: int | None) -> None:
    _check(_load().zero1_destroy(h))
    _HANDLES.pop(h, None)


def zero1_step(h: int, grad_ptrs, param_ptrs, stream=None) -> None:
    """One step: W device gradient buffers in, W device replicas out."""
    n, world, _ = _info(h)
    _check(_load().zero1_step(h, _ptrs(grad_ptrs, world, n, "bf16", True, "grads"),
                              _ptrs(param_ptrs, world, n, "bf16", True, "params"), _stream(stream)))


def zero1_step_host(h: int, host_grads, host_params, stream=None) -> None:
    """One step from host gradient buffers into host replica buffers (waits)."""
    n, world, _ = _info(h)
    _check(_load().zero1_step_host(h, _ptrs(host_grads, world, n, "bf16", False, "host_grads"),
                                   _ptrs(host_params, world, n, "bf16", False, "host_params"), _stream(stream)))


def zero1_step_host_async(h: int, host_grads, host_params, stream=None) -> None:
    """Pipelined host-buffer step; host_params are valid after zero1_host_sync."""
    n, world, _ = _info(h)
    _check(_load().zero1_step_host_async(h, _ptrs(host_grads, world, n, "bf16", False, "host_grads"),
                                         _ptrs(host_params, world, n, "bf16", False, "host_params"),
                                         _stream(stream)))


def zero1_host_sync(h: int) -> None:
    _check(_load().zero1_host_sync(h))


def _check_state(h, count, master, m, v) -> None:
    """master fp32, m and v fp32 (bf16 on a moments_bf16 handle), each able
    to hold `count` elements, in host or device memory."""
    if count is None:
        return
    mom = "bf16" if _info(h)[2] else "f32"
    _check_buffer(master, count, "f32", None, "master")
    _check_buffer(m, count, mom, None, "m")
    _check_buffer(v, count, mom, None, "v")


def zero1_set_state(h: int, master, m=None, v=None, t: int = 0, stream=None) -> None:
    _check_state(h, _info(h)[0], master, m, v)
    _check(_load().zero1_set_state(h, _addr(master), _addr(m), _addr(v), t, _stream(stream)))


def zero1_get_state(h: int, master=None, m=None, v=None, stream=None) -> int:
    _check_state(h, _info(h)[0], master, m, v)
    t = C.c_uint64()
    _check(_load().zero1_get_state(h, _addr(master), _addr(m), _addr(v), C.byref(t), _stream(stream)))
    return t.value


def zero1_set_state_range(h: int, offset: int, count: int, master, m=None, v=None, stream=None) -> None:
    _check_state(h, count, master, m, v)
    _check(_load().zero1_set_state_range(h, offset, count, _addr(master), _addr(m), _addr(v), _stream(stream)))


def zero1_get_state_range(h: int, offset: int, count: int, master=None, m=None, v=None, stream=None) -> None:
    _check_state(h, count, master, m, v)
    _check(_load().zero1_get_state_range(h, offset, count, _addr(master), _addr(m), _addr(v), _stream(stream)))


def zero1_set_lr(h: int, lr: float) -> None:
    _check(_load().zero1_set_lr(h, lr))


def zero1_set_lr_ptr(h: int, device_lr=None) -> None:
    """Capturable handles: read lr from a device float64 (None: own slot)."""
    _check(_load().zero1_set_lr_ptr(h, _addr(device_lr)))


def zero1_get_grad_norm(h: int, stream=None) -> tuple[float, float]:
    norm, clip = C.c_double(), C.c_float()
    _check(_load().zero1_get_grad_norm(h, C.byref(norm), C.byref(clip), _stream(stream)))
    return norm.value, clip.value


def zero1_layout(h: int) -> tuple[int, int, int]:
    s, p, b = C.c_uint64(), C.c_uint64(), C.c_uint64()
    _check(_load().zero1_layout(h, C.byref(s), C.byref(p), C.byref(b)))
    return s.value, p.value, b.value


def zero1_bucket_begin(h: int) -> None:
    _check(_load().zero1_bucket_begin(h))


def zero1_bucket_reduce(h: int, offset: int, count: int, grad_ptrs, stream=None) -> None:
    """Reduce-scatter one bucket: grad_ptrs[r] holds rank r's gradient for
    parameters [offset, offset+count)."""
    world = _info(h)[1]
    _check(_load().zero1_bucket_reduce(h, offset, count, _ptrs(grad_ptrs, world, count, "bf16", True, "grads"),
                                       _stream(stream)))


def zero1_bucket_update(h: int, offset: int, count: int, grad_ptrs, param_ptrs, stream=None) -> None:
    """Reduce-scatter and update one bucket (handles without clipping)."""
    world = _info(h)[1]
    _check(_load().zero1_bucket_update(h, offset, count, _ptrs(grad_ptrs, world, count, "bf16", True, "grads"),
                                       _ptrs(param_ptrs, world, count, "bf16", True, "params"), _stream(stream)))


def zero1_bucket_finish(h: int, param_ptrs, stream=None) -> None:
    n, world, _ = _info(h)
    table = None if param_ptrs is None else _ptrs(param_ptrs, world, n, "bf16", True, "params")
    _check(_load().zero1_bucket_finish(h, table, _stream(stream)))


def zero1_profile_start(h: int, capacity: int) -> None:
    _check(_load().zero1_profile_start(h, capacity))


def zero1_profile_stop(h: int) -> tuple[float, float, int]:
    """(summed reduce-scatter+norm ms, summed update+all-gather ms, steps)."""
    a, b, n = C.c_double(), C.c_double(), C.c_uint64()
    _check(_load().zero1_profile_stop(h, C.byref(a), C.byref(b), C.byref(n)))
    return a.value, b.value, n.value


def zero1_step_launches(h: int) -> int:
    """Kernel launches per zero1_step: 2, or 1 on the one-launch small-n path."""
    k = C.c_int()
    _check(_load().zero1_step_launches(h, C.byref(k)))
    return k.value


def zero1_profile_read(h: int, capacity: int) -> tuple[list[float], list[float]]:
    """Per-step (reduce-scatter+norm ms, update+all-gather ms) recorded so far."""
    a, b, n = (C.c_float * max(1, capacity))(), (C.c_float * max(1, capacity))(), C.c_uint64()
    _check(_load().zero1_profile_read(h, a, b, capacity, C.byref(n)))
    k = min(n.value, capacity)
    return list(a[:k]), list(b[:k])


def zero1_shard_plan(n: int, world: int) -> tuple[int, int]:
    """Shard length S and padded length W*S (host only, no device)."""
    s, p = C.c_uint64(), C.c_uint64()
    _check(_load().zero1_shard_plan(n, world, C.byref(s), C.byref(p)))
    return s.value, p.value


def zero1_step_scalars(hp: Hparams, world: int, t: int) -> dict:
    """The fp32 scalars step t uses (host only, no device)."""
    out = (C.c_float * 8)()
    c = hp._c()
    _check(_load().zero1_step_scalars(C.byref(c), world, t, out))
    keys = ("inv_w", "beta1", "one_minus_beta1", "beta2", "one_minus_beta2", "step_size", "decay", "eps")
    return dict(zip(keys, list(out)))


def zero1_step_noalloc(n: int, world: int, hp: Hparams, t: int, grad_ptrs, param_ptrs,
                       master, m, v, stream=None) -> None:
    """One step with caller-owned fp32 state and the library's fixed scratch
    (no device allocation; n <= 4,194,304)."""
    c = hp._c()
    grads = _ptrs(grad_ptrs, world, n, "bf16", True, "grads")
    params = _ptrs(param_ptrs, world, n, "bf16", True, "params")
    for x, name in ((master, "master"), (m, "m"), (v, "v")):
        _check_buffer(x, n, "f32", True, name)
    _check(_load().zero1_step_noalloc(n, world, C.byref(c), t, grads, params,
                                      _addr(master), _addr(m), _addr(v), _stream(stream)))


DTYPE_BF16, DTYPE_F32 = 0, 1
OP_SUM, OP_AVG = 0, 1


def zero1_allreduce(n: int, world: int, dtype: int, op: int, in_ptrs, out_ptrs, errors=None, stream=None) -> None:
    """DDP all-reduce of W device buffers (bf16 or fp32, sum or mean)."""
    kind = {DTYPE_BF16: "bf16", DTYPE_F32: "f32"}.get(dtype)
    _check(_load().zero1_allreduce(n, world, dtype, op, _ptrs(in_ptrs, world, n, kind, True, "in"),
                                   _ptrs(out_ptrs, world, n, kind, True, "out"), _addr(errors),
                                   _stream(stream)))


def zero1_allreduce_sum(h: int, in_ptrs, out_ptrs, stream=None) -> None:
    """bf16 sum all-reduce over the handle's W ranks of n elements each."""
    n, world, _ = _info(h)
    _check(_load().zero1_allreduce_sum(h, _ptrs(in_ptrs, world, n, "bf16", True, "in"),
                                       _ptrs(out_ptrs, world, n, "bf16", True, "out"), _stream(stream)))


def zero1_allgather(n: int, world: int, shard_len: int, dtype: int, shard_ptrs, out_ptrs, errors=None,
                    stream=None) -> None:
    """ZeRO-3 parameter all-gather: rank r's shard holds [r*S, min((r+1)*S, n))."""
    kind = {DTYPE_BF16: "bf16", DTYPE_F32: "f32"}.get(dtype)
    shards = _ptrs(shard_ptrs, world, None, None, True, "shards")
    if kind is not None and not isinstance(shard_ptrs, PtrTable):
        for r, x in enumerate(shard_ptrs):
            own = max(0, min(shard_len, n - r * shard_len))
            if own:
                _check_buffer(x, own, kind, True, f"shards[{r}]")
    _check(_load().zero1_allgather(n, world, shard_len, dtype, shards, _ptrs(out_ptrs, world, n, kind, True, "out"),
                                   _addr(errors), _stream(stream)))


# --------------------------------------------------------- matrices

SCALE_RMS, SCALE_SPECTRAL = 0, 1


class _CMatrix(C.Structure):
    _fields_ = [("offset", C.c_uint64), ("ld", C.c_uint64), ("rows", C.c_uint32), ("cols", C.c_uint32)]


class _CMuonHparams(C.Structure):
    _fields_ = [("size", C.c_uint32), ("nesterov", C.c_int32), ("scale_rule", C.c_int32), ("ns_steps", C.c_int32),
                ("lr", C.c_double), ("momentum", C.c_double), ("weight_decay", C.c_double), ("eps", C.c_double),
                ("update_scale", C.c_double), ("ns_a", C.c_double), ("ns_b", C.c_double), ("ns_c", C.c_double),
                ("inject_wait_timeout", C.c_int32), ("reserved", C.c_int32)]


@dataclass
class MuonHparams:
    """Hyperparameters of the matrix step (zero1_muon_hparams)."""
    lr: float = 1e-3
    momentum: float = 0.95
    weight_decay: float = 0.1
    eps: float = 1e-7
    update_scale: float = 0.2
    nesterov: bool = True
    scale_rule: int = SCALE_RMS
    ns_steps: int = 5
    ns_a: float = 3.4445
    ns_b: float = -4.7750
    ns_c: float = 2.0315
    inject_wait_timeout: bool = False    # failure testing: the tiled iteration's waits run out

    def _c(self) -> _CMuonHparams:
        return _CMuonHparams(C.sizeof(_CMuonHparams), int(self.nesterov), self.scale_rule, self.ns_steps, self.lr,
                             self.momentum, self.weight_decay, self.eps, self.update_scale, self.ns_a, self.ns_b,
                             self.ns_c, int(self.inject_wait_timeout), 0)


# (n, world) of every matrix handle this binding created.
_MUON_HANDLES: dict[int, tuple[int, int]] = {}


def _muon_info(h) -> tuple[int | None, int | None]:
    return _MUON_HANDLES.get(h, (None, None))


def zero1_muon_create(n: int, world: int, matrices, hp: MuonHparams | None = None) -> int:
    """Create a matrix handle; `matrices` holds (offset, rows, cols) or
    (offset, rows, cols, ld) tuples."""
    mats = [tuple(int(v) for v in m) for m in matrices]
    for i, m in enumerate(mats):
        if len(m) not in (3, 4):
            raise Zero1ArgumentError(f"matrices[{i}]: expected (offset, rows, cols[, ld]), got {m}")
        if any(v < 0 for v in m) or m[1] >= 1 << 32 or m[2] >= 1 << 32 or any(v >= 1 << 63 for v in m):
            raise Zero1ArgumentError(f"matrices[{i}]: {m} is out of range")
    table = (_CMatrix * max(1, len(mats)))(*[_CMatrix(m[0], m[3] if len(m) == 4 else m[2], m[1], m[2]) for m in mats])
    h = C.c_void_p()
    c = (hp or MuonHparams())._c()
    _check(_load().zero1_muon_create(n, world, table, len(mats), C.byref(c), C.byref(h)))
    _MUON_HANDLES[h.value] = (n, world)
    return h.value


def zero1_muon_destroy(h: int | None) -> None:
    _check(_load().zero1_muon_destroy(h))
    _MUON_HANDLES.pop(h, None)


def zero1_muon_step(h: int, grad_ptrs, param_ptrs, master, momentum, stream=None) -> None:
    """One step of the handle's matrices; master and momentum (fp32) are the
    caller's and are updated in place."""
    n, world = _muon_info(h)
    master = _addr(master) if n is None else _take(master, n, "f32", "master")
    momentum = _addr(momentum) if n is None else _take(momentum, n, "f32", "momentum")
    _check(_load().zero1_muon_step(h, _ptrs(grad_ptrs, world, n, "bf16", True, "grads"),
                                   _ptrs(param_ptrs, world, n, "bf16", True, "params"), master, momentum,
                                   _stream(stream)))


_KIND_OF = {DTYPE_BF16: "bf16", DTYPE_F32: "f32"}


def zero1_muon_orthogonalize(h: int, src, src_dtype: int, dst, dst_dtype: int, stream=None) -> None:
    """dst = the orthogonalised matrices of the flat buffer src."""
    n = _muon_info(h)[0]
    a, b = (_addr(x) if n is None or dtype not in _KIND_OF else _take(x, n, _KIND_OF[dtype], what)
            for x, dtype, what in ((src, src_dtype, "src"), (dst, dst_dtype, "dst")))
    _check(_load().zero1_muon_orthogonalize(h, a, src_dtype, b, dst_dtype, _stream(stream)))


def zero1_muon_set_lr(h: int, lr: float) -> None:
    _check(_load().zero1_muon_set_lr(h, lr))


def zero1_muon_status(h: int, stream=None) -> None:
    """Wait for the stream; raise if a kernel wait of this handle ever gave up."""
    _check(_load().zero1_muon_status(h, _stream(stream)))


def zero1_muon_layout(h: int) -> tuple[int, int]:
    """(entries of all matrices, device bytes the handle holds)."""
    e, b = C.c_uint64(), C.c_uint64()
    _check(_load().zero1_muon_layout(h, C.byref(e), C.byref(b)))
    return e.value, b.value


def _dtype_of(x, what: str) -> int:
    code = {"torch.bfloat16": DTYPE_BF16, "torch.float32": DTYPE_F32}.get(_dtype_name(x) if hasattr(x, "dtype") else "")
    if code is None:
        raise Zero1ArgumentError(f"{what}: expected a bf16 or fp32 tensor, got {getattr(x, 'dtype', type(x).__name__)}")
    return code


class Muon:
    """Owning wrapper around a matrix handle (closes on ``close()`` / context exit)."""

    def __init__(self, n: int, world: int, matrices, hp: MuonHparams | None = None):
        self.handle = None
        self.n, self.world, self.hp = n, world, hp or MuonHparams()
        self.handle = zero1_muon_create(n, world, matrices, self.hp)

    def step(self, grads, params, master, momentum, stream=None) -> None:
        zero1_muon_step(self.handle, grads, params, master, momentum, stream)

    def orthogonalize(self, src, dst, stream=None) -> None:
        """bf16 or fp32 tensors of n entries; the types may differ."""
        zero1_muon_orthogonalize(self.handle, src, _dtype_of(src, "src"), dst, _dtype_of(dst, "dst"), stream)

    def set_lr(self, lr: float) -> None:
        zero1_muon_set_lr(self.handle, lr)

    def status(self, stream=None) -> None:
        zero1_muon_status(self.handle, stream)

    def layout(self) -> tuple[int, int]:
        return zero1_muon_layout(self.handle)

    def close(self) -> None:
        if self.handle is not None:
            zero1_muon_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------- layer norm

def _take_rows(x, rows: int, cols: int, ld: int, kind: str | None, what: str) -> int | None:
    """Address of `x`, after refusing a torch tensor that is not CUDA memory of
    the type, has these rows at another stride than `ld`, or does not reach as
    far as rows `ld` apart do.  Raw addresses pass."""
    try:
        if x.dtype is _TORCH_DTYPES[kind] and x.is_cuda and x.shape == (rows, cols) and x.stride() == (ld, 1):
            return x.data_ptr()
    except (AttributeError, KeyError):
        pass
    if x is not None and hasattr(x, "data_ptr"):
        want = _KINDS[kind][0] if kind is not None else None
        if want is not None and _dtype_name(x) != want:
            raise Zero1ArgumentError(f"{what}: expected {want}, got {x.dtype}")
        if not x.is_cuda:
            raise Zero1ArgumentError(f"{what}: expected a CUDA tensor, got {x.device}")
        if rows:
            if x.dim() > 0 and x.stride(-1) != 1 and x.shape[-1] > 1:
                raise Zero1ArgumentError(f"{what}: the entries of a row must be adjacent")
            if rows > 1 and x.shape == (rows, cols) and x.stride(0) != ld:
                raise Zero1ArgumentError(f"{what}: its row stride is {x.stride(0)}, the call was given {ld}")
            held = x.untyped_storage().nbytes() // x.element_size() - x.storage_offset()
            if held < (rows - 1) * ld + cols:
                raise Zero1ArgumentError(f"{what}: its memory holds {held} elements, the call reads or writes "
                                         f"{(rows - 1) * ld + cols}")
    return _addr(x)


def _take_vector(x, count: int, kind: str | None, what: str) -> int | None:
    return _addr(x) if kind is None else _take(x, count, kind, what)


def zero1_layernorm_forward(rows: int, cols: int, dtype: int, x, ldx: int, gamma, beta, eps: float, y, ldy: int,
                            mean, rstd, stream=None) -> None:
    """y = layer norm of x; mean and rstd (fp32, one a row) for the backward pass."""
    kind = _KIND_OF.get(dtype)
    _check(_load().zero1_layernorm_forward(
        rows, cols, dtype, _take_rows(x, rows, cols, ldx, kind, "x"), ldx, _take_vector(gamma, cols, kind, "gamma"),
        _take_vector(beta, cols, kind, "beta"), eps, _take_rows(y, rows, cols, ldy, kind, "y"), ldy,
        _take(mean, rows, "f32", "mean"), _take(rstd, rows, "f32", "rstd"), _stream(stream)))


def zero1_layernorm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace the backward pass needs (host only, no device)."""
    b = C.c_uint64()
    _check(_load().zero1_layernorm_workspace(rows, cols, C.byref(b)))
    return b.value


def zero1_layernorm_backward(rows: int, cols: int, dtype: int, dy, lddy: int, x, ldx: int, gamma, mean, rstd, dx,
                             lddx: int, dgamma, dbeta, grad_dtype: int, workspace, stream=None) -> None:
    """dx, and the weight's and bias's gradients summed over all rows (bf16 or
    fp32); `workspace` is a CUDA tensor of at least zero1_layernorm_workspace
    bytes."""
    kind, grad_kind = _KIND_OF.get(dtype), _KIND_OF.get(grad_dtype)
    if not hasattr(workspace, "numel") or not workspace.is_cuda or not workspace.is_contiguous():
        raise Zero1ArgumentError("workspace: expected a contiguous CUDA tensor")
    _check(_load().zero1_layernorm_backward(
        rows, cols, dtype, _take_rows(dy, rows, cols, lddy, kind, "dy"), lddy,
        _take_rows(x, rows, cols, ldx, kind, "x"), ldx, _take_vector(gamma, cols, kind, "gamma"),
        _take(mean, rows, "f32", "mean"), _take(rstd, rows, "f32", "rstd"),
        _take_rows(dx, rows, cols, lddx, kind, "dx"), lddx, _take_vector(dgamma, cols, grad_kind, "dgamma"),
        _take_vector(dbeta, cols, grad_kind, "dbeta"), grad_dtype, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream)))


# --------------------------------------------------------- gated feed-forward block

ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = 0, 1, 2, 3


def _int32(v: int, what: str) -> int:
    """`v`, which C fields of 32 bits would otherwise cut off."""
    if not -(1 << 31) <= v < 1 << 31:
        raise Zero1ArgumentError(f"{what}: {v} is out of range")
    return v


class _CFfnShape(C.Structure):
    _fields_ = [("size", C.c_uint32), ("activation", C.c_int32)] + \
               [(k, C.c_uint64) for k in ("rows", "width", "hidden", "ldx", "ldy", "ldh", "ld_gate", "ld_up", "ld_down")] + \
               [("unaligned", C.c_int32), ("inject_wait_timeout", C.c_int32)]


@dataclass(frozen=True)
class FfnShape:
    """Sizes, activation and row strides of a gated feed-forward block (a
    stride of 0: rows one after another); `unaligned`: buffers need the
    alignment of their elements only."""
    rows: int
    width: int
    hidden: int
    activation: int = ACT_SILU
    ldx: int = 0
    ldy: int = 0
    ldh: int = 0
    ld_gate: int = 0
    ld_up: int = 0
    ld_down: int = 0
    unaligned: bool = False
    inject_wait_timeout: bool = False    # failure testing: the matrix kernels' waits run out

    def __post_init__(self):
        for k in ("rows", "width", "hidden", "ldx", "ldy", "ldh", "ld_gate", "ld_up", "ld_down"):
            if not 0 <= getattr(self, k) < 1 << 63:
                raise Zero1ArgumentError(f"{k}: {getattr(self, k)} is out of range")
        c = _CFfnShape(C.sizeof(_CFfnShape), _int32(self.activation, "activation"), self.rows, self.width, self.hidden,
                       self.ldx, self.ldy, self.ldh, self.ld_gate, self.ld_up, self.ld_down, int(self.unaligned),
                       int(self.inject_wait_timeout))
        r, w, h = self.rows, self.width, self.hidden
        # (rows, columns, stride, shape, strides) of x, y, h, w_gate, w_up and w_down, for the checks of every call
        mats = [(r, w, self.ldx or w), (r, w, self.ldy or w), (r, h, self.ldh or h), (w, h, self.ld_gate or h),
                (w, h, self.ld_up or h), (h, w, self.ld_down or w)]
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", C.byref(c))
        object.__setattr__(self, "_mats", [(a, b, ld, (a, b), (ld, 1)) for a, b, ld in mats])


def _take_matrix(x, matrix: tuple, what: str) -> int | None:
    """Address of the bf16 buffer `x` of a call, as _take_rows; a two-dimensional
    tensor has to be this matrix (rows, columns, stride, shape, strides)."""
    try:
        if x.dtype is _TORCH_DTYPES["bf16"] and x.is_cuda and x.shape == matrix[3] and x.stride() == matrix[4]:
            return x.data_ptr()
    except (AttributeError, KeyError):
        pass
    if x is not None and hasattr(x, "data_ptr") and x.dim() == 2 and x.shape != matrix[3]:
        raise Zero1ArgumentError(f"{what}: expected {matrix[0]} x {matrix[1]}, got {tuple(x.shape)}")
    return _take_rows(x, *matrix[:3], "bf16", what)


def _ffn_workspace(workspace) -> tuple[int | None, int]:
    if workspace is None:
        return None, 0
    try:
        if workspace.is_cuda and workspace.is_contiguous():
            return workspace.data_ptr() or None, workspace.nbytes
    except AttributeError:
        pass
    if not hasattr(workspace, "numel") or not workspace.is_cuda or not workspace.is_contiguous():
        raise Zero1ArgumentError("workspace: expected a contiguous CUDA tensor")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def _error_word(errors) -> int | None:
    """Address of the optional 32-bit word a kernel sets, which a tensor has to hold in device memory."""
    if errors is not None and hasattr(errors, "is_cuda"):
        if not errors.is_cuda:
            raise Zero1ArgumentError(f"errors: expected a CUDA tensor, got {errors.device}")
        if errors.nbytes < 4:
            raise Zero1ArgumentError(f"errors: {errors.nbytes} bytes, the call writes 4")
    return _addr(errors)


def zero1_ffn_workspace(shape: FfnShape, backward: bool = False) -> int:
    """Bytes of workspace a forward or backward call needs (host only, no device)."""
    b = C.c_uint64()
    _check(_load().zero1_ffn_workspace(C.byref(shape._c), int(backward), C.byref(b)))
    return b.value


def zero1_ffn_forward(shape: FfnShape, x, w_gate, w_up, w_down, gate, up, h, y, workspace=None, stream=None,
                      errors=None) -> None:
    """y = (act(x w_gate) * (x w_up)) w_down, keeping h and, unless both are
    None, gate and up; `workspace` is a CUDA tensor of at least
    zero1_ffn_workspace bytes, `errors` an optional CUDA word."""
    mx, my, mh, mg, mu, md = shape._mats
    rc = _load().zero1_ffn_forward(
        shape._ref, _take_matrix(x, mx, "x"), _take_matrix(w_gate, mg, "w_gate"), _take_matrix(w_up, mu, "w_up"),
        _take_matrix(w_down, md, "w_down"), None if gate is None else _take_matrix(gate, mh, "gate"),
        None if up is None else _take_matrix(up, mh, "up"), _take_matrix(h, mh, "h"), _take_matrix(y, my, "y"),
        *_ffn_workspace(workspace), _error_word(errors), _stream(stream))
    if rc:
        _check(rc)


def zero1_ffn_backward(shape: FfnShape, dy, x, w_gate, w_up, w_down, gate, up, h, dx, dw_gate, dw_up, dw_down,
                       workspace=None, stream=None, errors=None) -> None:
    """The gradients of x (None: not wanted) and of the three matrices, from the forward pass's gate, up and h."""
    mx, my, mh, mg, mu, md = shape._mats
    rc = _load().zero1_ffn_backward(
        shape._ref, _take_matrix(dy, my, "dy"), _take_matrix(x, mx, "x"), _take_matrix(w_gate, mg, "w_gate"),
        _take_matrix(w_up, mu, "w_up"), _take_matrix(w_down, md, "w_down"), _take_matrix(gate, mh, "gate"),
        _take_matrix(up, mh, "up"), _take_matrix(h, mh, "h"), None if dx is None else _take_matrix(dx, mx, "dx"),
        _take_matrix(dw_gate, mg, "dw_gate"), _take_matrix(dw_up, mu, "dw_up"), _take_matrix(dw_down, md, "dw_down"),
        *_ffn_workspace(workspace), _error_word(errors), _stream(stream))
    if rc:
        _check(rc)


# --------------------------------------------------------- AdamW over many tensors

class _CAdamWOptions(C.Structure):
    _fields_ = [("size", C.c_uint32), ("state_bits", C.c_int32), ("param_dtype", C.c_int32), ("grad_dtype", C.c_int32),
                ("decay_before_update", C.c_int32), ("reserved", C.c_int32), ("seed", C.c_uint64)]


@dataclass
class AdamWOptions:
    """Moments in 8 or 32 bits, the tensors' element types, torch's decay
    order, and the seed of the 8-bit codes' random rounding."""
    state_bits: int = 32
    param_dtype: int = DTYPE_BF16
    grad_dtype: int = DTYPE_BF16
    decay_before_update: bool = False
    seed: int = 0

    def _c(self) -> _CAdamWOptions:
        if not 0 <= self.seed < 1 << 64:
            raise Zero1ArgumentError(f"seed: {self.seed} is not an unsigned 64-bit number")
        ints = [_int32(getattr(self, k), k) for k in ("state_bits", "param_dtype", "grad_dtype")]
        return _CAdamWOptions(C.sizeof(_CAdamWOptions), *ints, int(self.decay_before_update), 0, self.seed)


# (sizes, a copy of the options, entries of the state) of every list handle this binding created.
_ADAMW_HANDLES: dict[int, tuple[tuple[int, ...], AdamWOptions, int]] = {}


def zero1_adamw_create(sizes, hp: Hparams | None = None, opts: AdamWOptions | None = None, decays=None) -> int:
    """Create a handle for tensors of these many entries; `decays` holds a
    truth value a tensor (None: all decay)."""
    # a copy: what the handle was created with, whatever becomes of the caller's object
    sizes, opts = tuple(int(n) for n in sizes), replace(opts or AdamWOptions())
    if any(not 0 <= n < 1 << 63 for n in sizes):
        raise Zero1ArgumentError("sizes: a size is out of range")
    if decays is not None:
        decays = [1 if d else 0 for d in decays]
        if len(decays) != len(sizes):
            raise Zero1ArgumentError(f"decays: {len(decays)} values given for {len(sizes)} tensors")
        decays = (C.c_uint8 * max(1, len(sizes)))(*decays)
    h = C.c_void_p()
    c, o = (hp or Hparams())._c(), opts._c()
    _check(_load().zero1_adamw_create((C.c_uint64 * max(1, len(sizes)))(*sizes), decays, len(sizes), C.byref(c),
                                      C.byref(o), C.byref(h)))
    _ADAMW_HANDLES[h.value] = (sizes, opts, sum(-(-n // 256) * 256 for n in sizes))
    return h.value


def zero1_adamw_destroy(h: int | None) -> None:
    _check(_load().zero1_adamw_destroy(h))
    _ADAMW_HANDLES.pop(h, None)


def _list_ptrs(xs, sizes, kind: str, what: str) -> C.Array:
    """The host array of one pointer a tensor, each checked to hold its
    tensor's entries."""
    if sizes is None:
        return xs.array if isinstance(xs, PtrTable) else (C.c_void_p * len(xs))(*[_addr(x) for x in xs])
    if len(xs) != len(sizes):
        raise Zero1ArgumentError(f"{what}: {len(xs)} pointers given, the call reads {len(sizes)}")
    if not isinstance(xs, PtrTable):
        return (C.c_void_p * len(sizes))(*[_take(x, n, kind, what, i) if n else None
                                           for i, (x, n) in enumerate(zip(xs, sizes))])
    key = (sizes, kind)
    if key not in xs._checked:
        for i, (x, n) in enumerate(zip(xs.buffers, sizes)):
            if n:
                _check_buffer(x, n, kind, True, f"{what}[{i}]")
        xs._checked.add(key)
    return xs.array


def _check_list_state(h, master, m, v, scales) -> tuple:
    """Addresses of the state buffers, after their checks."""
    _, opts, n = _ADAMW_HANDLES.get(h, (None, None, None))
    if n is None:
        return _addr(master), _addr(m), _addr(v), _addr(scales)
    kind = "u8" if opts.state_bits == 8 else "f32"
    return (_take(master, n, "f32", "master"), _take(m, n, kind, "m"), _take(v, n, kind, "v"),
            _take(scales, n // 128, "f32", "scales"))


def zero1_adamw_step(h: int, grad_ptrs, param_ptrs, master, m, v, scales=None, stream=None) -> None:
    """One step of all tensors; the state buffers are the caller's."""
    sizes, opts, _ = _ADAMW_HANDLES.get(h, (None, None, None))
    grads = _list_ptrs(grad_ptrs, sizes, _KIND_OF.get(opts.grad_dtype) if opts else None, "grads")
    params = _list_ptrs(param_ptrs, sizes, _KIND_OF.get(opts.param_dtype) if opts else None, "params")
    _check(_load().zero1_adamw_step(h, grads, params, *_check_list_state(h, master, m, v, scales), _stream(stream)))


def zero1_adamw_moments(h: int, m, v, scales, m_out=None, v_out=None, stream=None) -> None:
    """The fp32 values that 8-bit moments stand for."""
    n = _ADAMW_HANDLES.get(h, (None, None, None))[2]
    _, m, v, scales = _check_list_state(h, None, m, v, scales)
    outs = [_addr(x) if n is None else _take(x, n, "f32", what) for x, what in ((m_out, "m_out"), (v_out, "v_out"))]
    _check(_load().zero1_adamw_moments(h, m, v, scales, *outs, _stream(stream)))


def zero1_adamw_set_steps(h: int, t: int, stream=None) -> None:
    if not 0 <= t < 1 << 64:
        raise Zero1ArgumentError(f"steps: {t} is not an unsigned 64-bit number")
    _check(_load().zero1_adamw_set_steps(h, t, _stream(stream)))


def zero1_adamw_set_lr(h: int, lr: float, stream=None) -> None:
    _check(_load().zero1_adamw_set_lr(h, lr, _stream(stream)))


def zero1_adamw_get_steps(h: int, stream=None) -> int:
    t = C.c_uint64()
    _check(_load().zero1_adamw_get_steps(h, C.byref(t), _stream(stream)))
    return t.value


def zero1_adamw_get_grad_norm(h: int, stream=None) -> tuple[float, float]:
    norm, clip = C.c_double(), C.c_float()
    _check(_load().zero1_adamw_get_grad_norm(h, C.byref(norm), C.byref(clip), _stream(stream)))
    return norm.value, clip.value


def zero1_adamw_layout(h: int) -> tuple[int, list[int], int]:
    """(entries of each state buffer, where each tensor starts in them, device bytes of the handle)."""
    count = len(_ADAMW_HANDLES[h][0]) if h in _ADAMW_HANDLES else 0
    e, b, starts = C.c_uint64(), C.c_uint64(), (C.c_uint64 * max(1, count))()
    _check(_load().zero1_adamw_layout(h, C.byref(e), starts if count else None, C.byref(b)))
    return e.value, list(starts[:count]), b.value


class AdamW:
    """Owning wrapper around a list handle (closes on ``close()`` / context exit).

    ``entries`` is the length of master, m and v, ``scale_entries`` that of the
    8-bit moments' scales, and ``starts[i]`` where tensor i's state begins."""

    def __init__(self, sizes, hp: Hparams | None = None, opts: AdamWOptions | None = None, decays=None):
        self.handle = None
        self.hp, self.opts = replace(hp or Hparams()), replace(opts or AdamWOptions())
        self.handle = zero1_adamw_create(sizes, self.hp, self.opts, decays)
        self.entries, self.starts, _ = zero1_adamw_layout(self.handle)
        self.scale_entries = self.entries // 128 if self.opts.state_bits == 8 else 0

    def step(self, grads, params, master, m, v, scales=None, stream=None) -> None:
        zero1_adamw_step(self.handle, grads, params, master, m, v, scales, stream)

    def moments(self, m, v, scales, m_out=None, v_out=None, stream=None) -> None:
        zero1_adamw_moments(self.handle, m, v, scales, m_out, v_out, stream)

    def set_steps(self, t: int, stream=None) -> None:
        zero1_adamw_set_steps(self.handle, t, stream)

    def steps(self, stream=None) -> int:
        return zero1_adamw_get_steps(self.handle, stream)

    def set_lr(self, lr: float, stream=None) -> None:
        zero1_adamw_set_lr(self.handle, lr, stream)

    def grad_norm(self, stream=None) -> tuple[float, float]:
        return zero1_adamw_get_grad_norm(self.handle, stream)

    def layout(self) -> tuple[int, list[int], int]:
        return zero1_adamw_layout(self.handle)

    def close(self) -> None:
        if self.handle is not None:
            zero1_adamw_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _CSmPartition(C.Structure):
    _fields_ = [("stream_a", C.c_void_p), ("stream_b", C.c_void_p), ("sms_a", C.c_int), ("sms_b", C.c_int),
                ("opaque", C.c_void_p)]


def zero1_sm_partition_create(sms_a: int) -> _CSmPartition:
    """Two streams on disjoint SM groups of the current device (green
    contexts): the first with at least sms_a SMs, the second with the rest."""
    part = _CSmPartition()
    _check(_load().zero1_sm_partition_create(sms_a, C.byref(part)))
    return part


def zero1_sm_partition_destroy(part: _CSmPartition) -> None:
    _check(_load().zero1_sm_partition_destroy(C.byref(part)))


class SmPartition:
    """Owning wrapper of zero1_sm_partition_create: ``stream_a`` / ``stream_b``
    are the raw cudaStream_t values (wrap them with torch.cuda.ExternalStream),
    ``sms_a`` / ``sms_b`` the SMs each group was granted."""

    def __init__(self, sms_a: int):
        self._part = zero1_sm_partition_create(sms_a)
        self.stream_a, self.stream_b = self._part.stream_a, self._part.stream_b
        self.sms_a, self.sms_b = self._part.sms_a, self._part.sms_b

    def close(self) -> None:
        """Wait for both streams' work, then release the green contexts."""
        if self._part is not None:
            part, self._part = self._part, None
            zero1_sm_partition_destroy(part)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


class Zero1:
    """Owning wrapper around a handle (closes on ``close()`` / context exit)."""

    def __init__(self, n: int, world: int, hp: Hparams | None = None, opts: Options | None = None):
        self.n, self.world, self.hp, self.opts = n, world, hp or Hparams(), opts or Options()
        self.handle = zero1_create_ex(n, world, self.hp, self.opts)

    def step(self, grads, params, stream=None) -> None:
        zero1_step(self.handle, grads, params, stream)

    def step_host(self, grads, params, stream=None) -> None:
        zero1_step_host(self.handle, grads, params, stream)

    def step_host_async(self, grads, params, stream=None) -> None:
        zero1_step_host_async(self.handle, grads, params, stream)

    def host_sync(self) -> None:
        zero1_host_sync(self.handle)

    def launches_per_step(self) -> int:
        return zero1_step_launches(self.handle)

    def set_state(self, master, m=None, v=None, t: int = 0, stream=None) -> None:
        zero1_set_state(self.handle, master, m, v, t, stream)

    def get_state(self, master=None, m=None, v=None, stream=None) -> int:
        return zero1_get_state(self.handle, master, m, v, stream)

    def set_lr(self, lr: float) -> None:
        zero1_set_lr(self.handle, lr)

    def set_lr_ptr(self, device_lr=None) -> None:
        zero1_set_lr_ptr(self.handle, device_lr)

    def grad_norm(self, stream=None) -> tuple[float, float]:
        return zero1_get_grad_norm(self.handle, stream)

    def layout(self) -> tuple[int, int, int]:
        return zero1_layout(self.handle)

    def close(self) -> None:
        if self.handle is not None:
            zero1_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
