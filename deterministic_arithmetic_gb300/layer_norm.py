"""Layer norm, forward and backward (``lora_layer_norm_*`` of ``include/lora_mlp.h``).

``layer_norm_fwd(x, weight, bias)`` returns ``(y, mean, rstd)``; ``layer_norm_bwd(dy, x, weight,
mean, rstd)`` returns ``(dx, dw, db)`` and takes ``x`` as a tensor or as its 8-bit checkpoint
(``pack8.Packed8``). A row's results are the same bits in any batch; dw and db are the same bits
in every rerun. Every call takes ``stream=`` (default: the current stream). No autograd graph records
them. There is no fallback: without the library or off a GB300 the calls raise.
"""
from __future__ import annotations

from . import _capi as c


@c.on_stream
def layer_norm_fwd(x, weight, bias=None, eps: float = 1e-5, *, y=None, mean=None, rstd=None):
    """``y = (x - mean) * rstd * weight + bias`` over the rows of ``x`` [M, N] (bf16 or fp32).

    ``weight`` and ``bias`` (optional) are [N], both bf16 or both fp32; ``y`` has x's type,
    ``mean`` and ``rstd`` [M] are fp32 and kept for the backward pass."""
    return c.mlp.layer_norm_fwd(x, weight, bias, eps, y, mean, rstd)


def layer_norm_bwd_workspace_size(M: int, N: int) -> int:
    return c.fn("lora_layer_norm_bwd_workspace_size", (c.i64, c.i64), c.size_t)(M, N)


@c.on_stream
def layer_norm_bwd(dy, x, weight, mean, rstd, *, bias_grad: bool = True, dx=None, dw=None, db=None, workspace=None):
    """``(dx, dw, db)`` of ``dy`` [M, N]: ``dx`` of dy's type, ``dw`` and ``db`` [N] fp32 (``db``
    None when not ``bias_grad``). ``x`` is the forward's input, of dy's type, or its Packed8."""
    return c.mlp.layer_norm_bwd(dy, x, weight, mean, rstd, bias_grad, dx, dw, db, workspace)
