"""What the bindings of include/lora_mlp.h share: argument checks, the stream an operator runs on
and the allocation of what it returns. Argument marshalling only; the library does the work."""
from __future__ import annotations

import ctypes

import torch

from . import lora_delta as _ld

vp, i64, cint, f32, size_t = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
TYPE_CODES = {torch.bfloat16: 0, torch.float32: 1}

_fns: dict = {}


def fn(name: str, argtypes: tuple, restype=cint):
    """The entry point ``name`` of the library with its argument types set (looked up once)."""
    f = _fns.get(name)
    if f is None:
        f = getattr(_ld.library(), name)
        f.argtypes, f.restype = argtypes, restype
        _fns[name] = f
    return f


def check(t, name: str, shape: tuple, *dtypes, device=None):
    """``t`` is a contiguous CUDA tensor of one of ``dtypes`` and of ``shape`` (on ``device``)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {' or '.join(map(str, dtypes))} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ', not contiguous'}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: expected a tensor on {device or 'a CUDA device'}, got {t.device}")


def scratch(t, device):
    """(address, bytes) of a workspace tensor on ``device``."""
    if not t.is_contiguous() or t.device != device:
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def run_on(stream):
    """(handle, context) of the stream an operator runs on: memory allocated inside the context
    belongs to that stream, so a workspace is free again only behind the operator's kernels."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()), _NONE
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return int(stream.cuda_stream), torch.cuda.stream(stream)


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NONE = _Nothing()


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
