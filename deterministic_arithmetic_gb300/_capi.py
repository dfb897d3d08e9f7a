"""What the bindings of include/lora_mlp.h share: argument checks, outputs, the stream an operator runs
on. Argument marshalling only; the library does the work.

A small call costs more here than on the GPU (a launch takes about 2 us of host time, a checked and
allocating call about 12), so the checks read each property once, an output that was allocated here
is not checked again, and a stream other than the current one is entered by one wrapper."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import lora_delta as _ld

vp, i64, cint, f32, size_t = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
BF16, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8
TYPE_CODES = {BF16: 0, F32: 1}
empty = torch.empty

_fns: dict = {}


def fn(name: str, argtypes: tuple, restype=cint):
    """The entry point ``name`` of the library with its argument types set (looked up once)."""
    f = _fns.get(name)
    if f is None:
        f = getattr(_ld.library(), name)
        f.argtypes, f.restype = argtypes, restype
        _fns[name] = f
    return f


def _refuse(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    where = "a CUDA device" if device is None or device < 0 else f"cuda:{device}"
    raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} {tuple(shape)} on {where}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def check(t, name: str, shape: tuple, dtype, device: int) -> int:
    """The address of ``t``, a contiguous tensor of ``dtype`` and ``shape`` on CUDA device ``device``."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and device >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, (dtype,), device)


def check_either(t, name: str, shape: tuple, device: int) -> int:
    """The same for a bf16 or fp32 tensor."""
    return check(t, name, shape, F32 if getattr(t, "dtype", None) is F32 else BF16, device)


def device_of(t, name: str) -> int:
    """The CUDA device an operator runs on: that of its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t.get_device()


def out(t, name: str, shape: tuple, dtype, device: int):
    """An output: the caller's tensor, checked, or a new one."""
    if t is None:
        return empty(shape, dtype=dtype, device=device)
    check(t, name, shape, dtype, device)
    return t


def scratch(t, device: int):
    """(address, bytes) of a workspace tensor on ``device``."""
    if not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{device}, got one on {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def stream(device: int) -> int:
    """Handle of the current stream of ``device``."""
    return torch._C._cuda_getCurrentRawStream(device)


def on_stream(f):
    """Gives ``f`` the argument ``stream`` (a torch stream or a handle; None: the current one). ``f`` runs
    with that stream current, so that memory it allocates belongs to the stream: a workspace is free
    again only behind the operator's kernels."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def done(rc: int, name: str):
    if rc:
        raise _ld.LoraDeltaError(rc, name)


def device_status() -> int:
    """Code that a kernel of include/lora_mlp.h left when it gave up on a wait, or 0 (synchronises)."""
    code = cint(0)
    rc = fn("lora_mlp_device_status", (ctypes.POINTER(cint),))(ctypes.byref(code))
    if rc not in (0, 8):
        raise _ld.LoraDeltaError(rc, "lora_mlp_device_status")
    return code.value


def device_status_reset(stall_kind: int = 0, wait_limit_us: int = 0) -> None:
    """Clear that code (synchronises); the arguments are for tests (include/lora_mlp.h)."""
    done(fn("lora_mlp_device_status_reset", (cint, cint))(stall_kind, wait_limit_us), "lora_mlp_device_status_reset")
