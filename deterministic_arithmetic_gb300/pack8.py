"""Activation checkpoints in 8 bits (``lora_pack8``, ``lora_unpack8`` and the backward passes from
packed activations of ``include/lora_mlp.h``).

A ``Packed8`` holds int8 codes and one scale byte per group of 32 elements of a row; a code times
its power-of-two step is a bf16 value exactly, so a backward pass from the checkpoint gives bit for
bit what it gives for the unpacked tensor. Every call takes ``stream=`` (default: the current
stream). No autograd graph records them. There is no fallback.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _capi as c

GROUP = 32
_TYPE_CODES = {torch.bfloat16: 0, torch.float32: 1}


@dataclass(slots=True)
class Packed8:
    """A [rows, cols] activation in 8 bits: ``codes`` [rows, 32 * groups] int8 (zero past ``cols``),
    ``scales`` [rows, groups] uint8, groups = ceil(cols / 32)."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


@c.on_stream
def pack8(x, *, out: Packed8 | None = None) -> Packed8:
    """The 8-bit form of ``x`` [M, K] (bf16 or fp32)."""
    return c.mlp.pack8(x, out)


@c.on_stream
def unpack8(p: Packed8, *, dtype=torch.bfloat16, out=None):
    """The values ``p`` stands for, [M, K] bf16 (exact) or fp32."""
    code = _TYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"unpack8: values of torch.bfloat16 or torch.float32, not {dtype}")
    return c.mlp.unpack8(p, code, out)


def pack8_da_workspace_size(M: int, K: int, R: int) -> int:
    return c.fn("lora_pack8_da_workspace_size", (c.i64,) * 3, c.size_t)(M, K, R)


@c.on_stream
def pack8_da(du, p: Packed8, *, da=None, workspace=None):
    """``dA = du.T @ x`` (fp32 [R, K]) of a packed ``x``: ``du`` [M, R] bf16. Bit for bit the dA of
    ``lora_delta_bwd`` for the unpacked x."""
    return c.mlp.pack8_da(du, p, da, workspace)


def lora_delta_bwd_packed8_workspace_size(M: int, K: int, N: int, R: int) -> int:
    return c.fn("lora_delta_bwd_packed8_workspace_size", (c.i64,) * 4, c.size_t)(M, K, N, R)


@c.on_stream
def lora_delta_bwd_packed8(dy, p: Packed8, a, b, u, alpha: float, *, dx=None, da=None, db=None, du=None,
                           workspace=None):
    """``lora_delta.lora_delta_bwd(dy, x, a, b, u, alpha)`` with x given as its 8-bit checkpoint:
    ``(dx, da, db, du)``, bit for bit those of the unpacked x; of no rows, ``da`` and ``db`` are zeros.
    ``workspace`` (optional): ``lora_delta.new_workspace`` of the size above."""
    return c.mlp.lora_delta_bwd_packed8(dy, p, a, b, u, alpha, dx, da, db, du, workspace)
