"""Layer norm, forward and backward (``lora_layer_norm_*`` of ``include/lora_mlp.h``).

``layer_norm_fwd(x, weight, bias)`` returns ``(y, mean, rstd)``; ``layer_norm_bwd(dy, x, weight,
mean, rstd)`` returns ``(dx, dw, db)`` and takes ``x`` as a tensor or as its 8-bit checkpoint
(``pack8.Packed8``). A row's results are the same bits in any batch; dw and db are the same bits
in every rerun. There is no fallback: without the library or off a GB300 the calls raise.
"""
from __future__ import annotations

import torch

from . import _capi as c
from .pack8 import Packed8, check_packed

_FWD = (c.vp, c.cint, c.vp, c.vp, c.cint, c.f32, c.i64, c.i64, c.vp, c.vp, c.vp, c.vp)
_BWD = (c.vp, c.cint, c.vp, c.vp, c.vp, c.cint, c.vp, c.vp, c.i64, c.i64, c.vp, c.vp, c.vp, c.vp, c.size_t, c.vp)


def layer_norm_fwd(x, weight, bias=None, eps: float = 1e-5, *, y=None, mean=None, rstd=None, stream=None):
    """``y = (x - mean) * rstd * weight + bias`` over the rows of ``x`` [M, N] (bf16 or fp32).

    ``weight`` and ``bias`` (optional) are [N], both bf16 or both fp32; ``y`` has x's type,
    ``mean`` and ``rstd`` [M] are fp32 and kept for the backward pass."""
    M, N = x.shape
    c.check(x, "x", (M, N), torch.bfloat16, torch.float32)
    c.check(weight, "weight", (N,), torch.bfloat16, torch.float32, device=x.device)
    if bias is not None:
        c.check(bias, "bias", (N,), weight.dtype, device=x.device)
    handle, on = c.run_on(stream)
    with on:
        y = torch.empty_like(x) if y is None else y
        mean = torch.empty(M, dtype=torch.float32, device=x.device) if mean is None else mean
        rstd = torch.empty(M, dtype=torch.float32, device=x.device) if rstd is None else rstd
    c.check(y, "y", (M, N), x.dtype, device=x.device)
    c.check(mean, "mean", (M,), torch.float32, device=x.device)
    c.check(rstd, "rstd", (M,), torch.float32, device=x.device)
    c.done(c.fn("lora_layer_norm_fwd", _FWD)(
        x.data_ptr(), c.TYPE_CODES[x.dtype], weight.data_ptr(), None if bias is None else bias.data_ptr(),
        c.TYPE_CODES[weight.dtype], eps, M, N, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), handle),
        "lora_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd_workspace_size(M: int, N: int) -> int:
    return int(c.fn("lora_layer_norm_bwd_workspace_size", (c.i64, c.i64), c.size_t)(M, N))


def layer_norm_bwd(dy, x, weight, mean, rstd, *, bias_grad: bool = True, dx=None, dw=None, db=None, workspace=None,
                   stream=None):
    """``(dx, dw, db)`` of ``dy`` [M, N]: ``dx`` of dy's type, ``dw`` and ``db`` [N] fp32 (``db``
    None when not ``bias_grad``). ``x`` is the forward's input, of dy's type, or its Packed8."""
    M, N = dy.shape
    c.check(dy, "dy", (M, N), torch.bfloat16, torch.float32)
    dev = dy.device
    if isinstance(x, Packed8):
        check_packed(x, "x", M, N, dev)
        x_ptr, scales_ptr = x.codes.data_ptr(), x.scales.data_ptr()
    else:
        c.check(x, "x", (M, N), dy.dtype, device=dev)
        x_ptr, scales_ptr = x.data_ptr(), None
    c.check(weight, "weight", (N,), torch.bfloat16, torch.float32, device=dev)
    c.check(mean, "mean", (M,), torch.float32, device=dev)
    c.check(rstd, "rstd", (M,), torch.float32, device=dev)
    handle, on = c.run_on(stream)
    with on:
        dx = torch.empty_like(dy) if dx is None else dx
        dw = torch.empty(N, dtype=torch.float32, device=dev) if dw is None else dw
        if bias_grad and db is None:
            db = torch.empty(N, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(layer_norm_bwd_workspace_size(M, N), dtype=torch.uint8, device=dev)
    c.check(dx, "dx", (M, N), dy.dtype, device=dev)
    c.check(dw, "dw", (N,), torch.float32, device=dev)
    if bias_grad:
        c.check(db, "db", (N,), torch.float32, device=dev)
    c.done(c.fn("lora_layer_norm_bwd", _BWD)(
        dy.data_ptr(), c.TYPE_CODES[dy.dtype], x_ptr, scales_ptr, weight.data_ptr(), c.TYPE_CODES[weight.dtype],
        mean.data_ptr(), rstd.data_ptr(), M, N, dx.data_ptr(), dw.data_ptr(), db.data_ptr() if bias_grad else None,
        *c.scratch(workspace, dev), handle), "lora_layer_norm_bwd")
    return dx, dw, db if bias_grad else None
