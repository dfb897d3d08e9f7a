"""Tensors in 8-bit blocks of 128 and the products with weights held so (``lora_block8*`` of
``include/lora_base8.h``): a frozen base layer at a byte a weight.

A ``Block8`` holds e4m3 codes and an FP32 scale for each block of ``tile`` rows by 128 columns: tile 1 for
activations and gradients, 128 for weights. ``block8`` chooses power-of-two scales, and every value it then stands
for is a bf16 value exactly; the products take any scales. One copy of a weight's codes serves both passes.
A row's results are the same bits in any batch. Every call takes ``stream=`` (default: the current stream). No
autograd graph records them. There is no fallback.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _capi as c

BLOCK = 128
_TYPE_CODES = {torch.bfloat16: 0, torch.float32: 1}


@dataclass(slots=True)
class Block8:
    """A [rows, cols] tensor in 8-bit blocks: ``codes`` [rows, 16 * ceil(cols / 16)] float8_e4m3fn (not read past
    ``cols``), ``scales`` [ceil(rows / tile), ceil(cols / 128)] fp32, ``tile`` 1 or 128."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int
    tile: int = 1


def _code(dtype, name: str) -> int:
    code = _TYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"{name}: torch.bfloat16 or torch.float32, not {dtype}")
    return code


@c.on_stream
def block8(x, *, tile: int = 1, out: Block8 | None = None) -> Block8:
    """The 8-bit form of ``x`` [M, K] (bf16 or fp32): a scale for each 128 elements of a row (``tile`` 1), or for each
    128 x 128 (``tile`` 128, a weight). A block with a NaN or an infinity reads NaN."""
    return c.mlp.block8(x, tile, out)


@c.on_stream
def unblock8(p: Block8, *, dtype=torch.bfloat16, out=None):
    """The values ``p`` stands for, [M, K] bf16 or fp32."""
    return c.mlp.unblock8(p, _code(dtype, "dtype"), out)


@c.on_stream
def block8_linear_fwd(x: Block8, w: Block8, *, delta=None, dtype=torch.bfloat16, y=None):
    """``y = x @ w.T + delta`` [M, N]: ``x`` [M, K] of tile 1, ``w`` [N, K] of tile 128, ``delta`` fp32 [M, N] (the
    adapter's, from ``lora_delta_fwd``) or None; ``y`` bf16 or fp32, rounded once."""
    return c.mlp.block8_linear_fwd(x, w, delta, _code(dtype, "dtype"), y)


@c.on_stream
def block8_linear_bwd(dy: Block8, w: Block8, *, delta=None, dtype=torch.bfloat16, dx=None):
    """``dx = dy @ w + delta`` [M, K]: ``dy`` [M, N] of tile 1, the forward's ``w``, ``delta`` fp32 [M, K] (the
    adapter's dx, from ``lora_delta_bwd``) or None. The weight is frozen: it has no gradient."""
    return c.mlp.block8_linear_bwd(dy, w, delta, _code(dtype, "dtype"), dx)
