"""What the Python modules over include/lora_mlp.h and include/lora_base8.h share: the compiled binding ``_mlp``, entry points of
the C ABI for what needs no tensors, and the choice of stream."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import lora_delta as _ld

vp, i64, cint, f32, size_t = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

_fns: dict = {}


def fn(name: str, argtypes: tuple, restype=cint):
    """The entry point ``name`` of the library with its argument types set (looked up once)."""
    f = _fns.get(name)
    if f is None:
        f = getattr(_ld.library(), name)
        f.argtypes, f.restype = argtypes, restype
        _fns[name] = f
    return f


class _Binding:
    """The compiled binding, loaded (after the library it calls) when an operator is first called."""

    def __getattr__(self, name):
        _ld.library()
        from . import _mlp
        from .block8 import Block8
        from .pack8 import Packed8

        _mlp.setup(Packed8, Block8, _ld.LoraDeltaError)
        for f in dir(_mlp):
            if not f.startswith("_"):
                setattr(self, f, getattr(_mlp, f))
        return getattr(_mlp, name)


mlp = _Binding()


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


def device_status() -> int:
    """Code that a kernel of include/lora_mlp.h left when it gave up on a wait, or 0 (synchronises)."""
    code = cint(0)
    rc = fn("lora_mlp_device_status", (ctypes.POINTER(cint),))(ctypes.byref(code))
    if rc not in (0, 8):
        raise _ld.LoraDeltaError(rc, "lora_mlp_device_status")
    return code.value


def device_status_reset(stall_kind: int = 0, wait_limit_us: int = 0) -> None:
    """Clear that code (synchronises); the arguments are for tests (include/lora_mlp.h)."""
    rc = fn("lora_mlp_device_status_reset", (cint, cint))(stall_kind, wait_limit_us)
    if rc:
        raise _ld.LoraDeltaError(rc, "lora_mlp_device_status_reset")
