"""Activation checkpoints in 8 bits (``lora_pack8``, ``lora_unpack8`` and the backward passes from
packed activations of ``include/lora_mlp.h``).

A ``Packed8`` holds int8 codes and one scale byte per group of 32 elements of a row; a code times
its power-of-two step is a bf16 value exactly, so a backward pass from the checkpoint gives bit for
bit what it gives for the unpacked tensor. Every call takes ``stream=`` (default: the current
stream). There is no fallback.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _capi as c
from . import lora_delta as _ld

GROUP = 32

_PACK = (c.vp, c.cint, c.i64, c.i64, c.vp, c.vp, c.vp)
_UNPACK = (c.vp, c.vp, c.i64, c.i64, c.vp, c.cint, c.vp)
_DA = (c.vp, c.vp, c.vp, c.i64, c.i64, c.i64, c.vp, c.vp, c.size_t, c.vp)
_BWD = (c.vp,) * 6 + (c.f32,) + (c.i64,) * 4 + (c.vp,) * 5 + (c.size_t, c.vp)


@dataclass(slots=True)
class Packed8:
    """A [rows, cols] activation in 8 bits: ``codes`` [rows, 32 * groups] int8 (zero past ``cols``),
    ``scales`` [rows, groups] uint8."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


def groups(cols: int) -> int:
    """Scale bytes of a row of ``cols`` elements."""
    return -(-cols // GROUP)


def _cols(p, name: str) -> int:
    if not isinstance(p, Packed8):
        raise TypeError(f"{name} must be a Packed8")
    return p.cols


def check_packed(p: Packed8, name: str, rows: int, cols: int, device: int) -> tuple[int, int]:
    """The addresses of the codes and scales of a Packed8 of that size."""
    _cols(p, name)
    if p.cols != cols:
        raise ValueError(f"{name}: expected {cols} columns, got {p.cols}")
    g = -(-cols // GROUP)
    return (c.check(p.codes, name + ".codes", (rows, GROUP * g), c.I8, device),
            c.check(p.scales, name + ".scales", (rows, g), c.U8, device))


def new_packed(rows: int, cols: int, device: int) -> Packed8:
    g = groups(cols)
    return Packed8(c.empty((rows, GROUP * g), dtype=c.I8, device=device), c.empty((rows, g), dtype=c.U8, device=device),
                   cols)


@c.on_stream
def pack8(x, *, out: Packed8 | None = None) -> Packed8:
    """The 8-bit form of ``x`` [M, K] (bf16 or fp32)."""
    dev = c.device_of(x, "x")
    M, K = x.shape
    xp = c.check_either(x, "x", x.shape, dev)
    if out is None:
        out = new_packed(M, K, dev)
        cp, sp = out.codes.data_ptr(), out.scales.data_ptr()
    else:
        cp, sp = check_packed(out, "out", M, K, dev)
    c.done(c.fn("lora_pack8", _PACK)(xp, c.TYPE_CODES[x.dtype], M, K, cp, sp, c.stream(dev)), "lora_pack8")
    return out


@c.on_stream
def unpack8(p: Packed8, *, dtype=torch.bfloat16, out=None):
    """The values ``p`` stands for, [M, K] bf16 (exact) or fp32."""
    K = _cols(p, "p")
    dev, M = c.device_of(p.codes, "p.codes"), p.codes.shape[0]
    cp, sp = check_packed(p, "p", M, K, dev)
    if out is not None:
        dtype = out.dtype
    if dtype not in c.TYPE_CODES:
        raise ValueError(f"unpack8: values of torch.bfloat16 or torch.float32, not {dtype}")
    out = c.out(out, "out", (M, K), dtype, dev)
    c.done(c.fn("lora_unpack8", _UNPACK)(cp, sp, M, K, out.data_ptr(), c.TYPE_CODES[dtype], c.stream(dev)),
           "lora_unpack8")
    return out


def pack8_da_workspace_size(M: int, K: int, R: int) -> int:
    return c.fn("lora_pack8_da_workspace_size", (c.i64,) * 3, c.size_t)(M, K, R)


@c.on_stream
def pack8_da(du, p: Packed8, *, da=None, workspace=None):
    """``dA = du.T @ x`` (fp32 [R, K]) of a packed ``x``: ``du`` [M, R] bf16. Bit for bit the dA of
    ``lora_delta_bwd`` for the unpacked x."""
    dev = c.device_of(du, "du")
    M, R = du.shape
    dup = c.check(du, "du", du.shape, c.BF16, dev)
    K = _cols(p, "p")
    cp, sp = check_packed(p, "p", M, K, dev)
    da = c.out(da, "da", (R, K), c.F32, dev)
    if workspace is None:
        workspace = c.empty(pack8_da_workspace_size(M, K, R), dtype=c.U8, device=dev)
    c.done(c.fn("lora_pack8_da", _DA)(dup, cp, sp, M, K, R, da.data_ptr(), *c.scratch(workspace, dev), c.stream(dev)),
           "lora_pack8_da")
    return da


def lora_delta_bwd_packed8_workspace_size(M: int, K: int, N: int, R: int) -> int:
    return c.fn("lora_delta_bwd_packed8_workspace_size", (c.i64,) * 4, c.size_t)(M, K, N, R)


@c.on_stream
def lora_delta_bwd_packed8(dy, p: Packed8, a, b, u, alpha: float, *, dx=None, da=None, db=None, du=None,
                           workspace=None):
    """``lora_delta.lora_delta_bwd(dy, x, a, b, u, alpha)`` with x given as its 8-bit checkpoint:
    ``(dx, da, db, du)``, bit for bit those of the unpacked x. ``workspace`` (optional):
    ``lora_delta.new_workspace`` of the size above."""
    dev = c.device_of(dy, "dy")
    M, N = dy.shape
    K, R = _cols(p, "p"), a.shape[0]
    dyp = c.check(dy, "dy", (M, N), c.BF16, dev)
    cp, sp = check_packed(p, "p", M, K, dev)
    ap, bp = c.check(a, "a", (R, K), c.BF16, dev), c.check(b, "b", (N, R), c.BF16, dev)
    up = c.check(u, "u", (M, R), c.BF16, dev)
    dx = c.out(dx, "dx", (M, K), c.F32, dev)
    da = c.out(da, "da", (R, K), c.F32, dev)
    db = c.out(db, "db", (N, R), c.F32, dev)
    du = c.out(du, "du", (M, R), c.BF16, dev)
    if workspace is None:
        workspace = _ld.new_workspace(lora_delta_bwd_packed8_workspace_size(M, K, N, R), dy.device)
    c.done(c.fn("lora_delta_bwd_packed8", _BWD)(
        dyp, cp, sp, ap, bp, up, float(alpha), M, K, N, R, dx.data_ptr(), da.data_ptr(), db.data_ptr(), du.data_ptr(),
        *c.scratch(workspace, dev), c.stream(dev)), "lora_delta_bwd_packed8")
    return dx, da, db, du
