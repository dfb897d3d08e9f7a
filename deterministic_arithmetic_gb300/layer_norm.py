"""Layer norm, forward and backward (``lora_layer_norm_*`` of ``include/lora_mlp.h``).

``layer_norm_fwd(x, weight, bias)`` returns ``(y, mean, rstd)``; ``layer_norm_bwd(dy, x, weight,
mean, rstd)`` returns ``(dx, dw, db)`` and takes ``x`` as a tensor or as its 8-bit checkpoint
(``pack8.Packed8``). A row's results are the same bits in any batch; dw and db are the same bits
in every rerun. Every call takes ``stream=`` (default: the current stream). There is no fallback:
without the library or off a GB300 the calls raise.
"""
from __future__ import annotations

from . import _capi as c
from .pack8 import Packed8, check_packed

_FWD = (c.vp, c.cint, c.vp, c.vp, c.cint, c.f32, c.i64, c.i64, c.vp, c.vp, c.vp, c.vp)
_BWD = (c.vp, c.cint, c.vp, c.vp, c.vp, c.cint, c.vp, c.vp, c.i64, c.i64, c.vp, c.vp, c.vp, c.vp, c.size_t, c.vp)


@c.on_stream
def layer_norm_fwd(x, weight, bias=None, eps: float = 1e-5, *, y=None, mean=None, rstd=None):
    """``y = (x - mean) * rstd * weight + bias`` over the rows of ``x`` [M, N] (bf16 or fp32).

    ``weight`` and ``bias`` (optional) are [N], both bf16 or both fp32; ``y`` has x's type,
    ``mean`` and ``rstd`` [M] are fp32 and kept for the backward pass."""
    dev = c.device_of(x, "x")
    M, N = shape = x.shape
    xp = c.check_either(x, "x", shape, dev)
    wp = c.check_either(weight, "weight", (N,), dev)
    bp = None if bias is None else c.check(bias, "bias", (N,), weight.dtype, dev)
    y = c.out(y, "y", shape, x.dtype, dev)
    mean = c.out(mean, "mean", (M,), c.F32, dev)
    rstd = c.out(rstd, "rstd", (M,), c.F32, dev)
    c.done(c.fn("lora_layer_norm_fwd", _FWD)(
        xp, c.TYPE_CODES[x.dtype], wp, bp, c.TYPE_CODES[weight.dtype], eps, M, N, y.data_ptr(), mean.data_ptr(),
        rstd.data_ptr(), c.stream(dev)), "lora_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_bwd_workspace_size(M: int, N: int) -> int:
    return c.fn("lora_layer_norm_bwd_workspace_size", (c.i64, c.i64), c.size_t)(M, N)


@c.on_stream
def layer_norm_bwd(dy, x, weight, mean, rstd, *, bias_grad: bool = True, dx=None, dw=None, db=None, workspace=None):
    """``(dx, dw, db)`` of ``dy`` [M, N]: ``dx`` of dy's type, ``dw`` and ``db`` [N] fp32 (``db``
    None when not ``bias_grad``). ``x`` is the forward's input, of dy's type, or its Packed8."""
    dev = c.device_of(dy, "dy")
    M, N = shape = dy.shape
    dyp = c.check_either(dy, "dy", shape, dev)
    if isinstance(x, Packed8):
        xp, xs = check_packed(x, "x", M, N, dev)
    else:
        xp, xs = c.check(x, "x", shape, dy.dtype, dev), None
    wp = c.check_either(weight, "weight", (N,), dev)
    mp, rp = c.check(mean, "mean", (M,), c.F32, dev), c.check(rstd, "rstd", (M,), c.F32, dev)
    dx = c.out(dx, "dx", shape, dy.dtype, dev)
    dw = c.out(dw, "dw", (N,), c.F32, dev)
    db = c.out(db, "db", (N,), c.F32, dev) if bias_grad else None
    if workspace is None:
        workspace = c.empty(layer_norm_bwd_workspace_size(M, N), dtype=c.U8, device=dev)
    c.done(c.fn("lora_layer_norm_bwd", _BWD)(
        dyp, c.TYPE_CODES[dy.dtype], xp, xs, wp, c.TYPE_CODES[weight.dtype], mp, rp, M, N, dx.data_ptr(), dw.data_ptr(),
        db.data_ptr() if bias_grad else None, *c.scratch(workspace, dev), c.stream(dev)), "lora_layer_norm_bwd")
    return dx, dw, db
