"""Activation checkpoints in 8 bits (``lora_pack8``, ``lora_unpack8`` and the backward passes from
packed activations of ``include/lora_mlp.h``).

A ``Packed8`` holds int8 codes and one scale byte per group of 32 elements of a row; a code times
its power-of-two step is a bf16 value exactly, so a backward pass from the checkpoint gives bit for
bit what it gives for the unpacked tensor. There is no fallback.
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


@dataclass(frozen=True)
class Packed8:
    """A [rows, cols] activation in 8 bits: ``codes`` [rows, 32 * groups] int8 (zero past ``cols``),
    ``scales`` [rows, groups] uint8."""
    codes: torch.Tensor
    scales: torch.Tensor
    cols: int


def groups(cols: int) -> int:
    """Scale bytes of a row of ``cols`` elements."""
    return -(-cols // GROUP)


def _is_packed(p, name: str):
    if not isinstance(p, Packed8):
        raise TypeError(f"{name} must be a Packed8")


def check_packed(p: Packed8, name: str, rows: int, cols: int, device):
    _is_packed(p, name)
    if p.cols != cols:
        raise ValueError(f"{name}: expected {cols} columns, got {p.cols}")
    g = groups(cols)
    c.check(p.codes, name + ".codes", (rows, GROUP * g), torch.int8, device=device)
    c.check(p.scales, name + ".scales", (rows, g), torch.uint8, device=device)


def new_packed(rows: int, cols: int, device) -> Packed8:
    g = groups(cols)
    return Packed8(torch.empty((rows, GROUP * g), dtype=torch.int8, device=device),
                   torch.empty((rows, g), dtype=torch.uint8, device=device), cols)


def pack8(x, *, out: Packed8 | None = None, stream=None) -> Packed8:
    """The 8-bit form of ``x`` [M, K] (bf16 or fp32)."""
    M, K = x.shape
    c.check(x, "x", (M, K), torch.bfloat16, torch.float32)
    handle, on = c.run_on(stream)
    with on:
        out = new_packed(M, K, x.device) if out is None else out
    check_packed(out, "out", M, K, x.device)
    c.done(c.fn("lora_pack8", _PACK)(x.data_ptr(), c.TYPE_CODES[x.dtype], M, K, out.codes.data_ptr(),
                                     out.scales.data_ptr(), handle), "lora_pack8")
    return out


def unpack8(p: Packed8, *, dtype=torch.bfloat16, out=None, stream=None):
    """The values ``p`` stands for, [M, K] bf16 (exact) or fp32."""
    _is_packed(p, "p")
    M, K = p.codes.shape[0], p.cols
    check_packed(p, "p", M, K, p.codes.device)
    handle, on = c.run_on(stream)
    with on:
        out = torch.empty((M, K), dtype=dtype, device=p.codes.device) if out is None else out
    c.check(out, "out", (M, K), torch.bfloat16, torch.float32, device=p.codes.device)
    c.done(c.fn("lora_unpack8", _UNPACK)(p.codes.data_ptr(), p.scales.data_ptr(), M, K, out.data_ptr(),
                                         c.TYPE_CODES[out.dtype], handle), "lora_unpack8")
    return out


def pack8_da_workspace_size(M: int, K: int, R: int) -> int:
    return int(c.fn("lora_pack8_da_workspace_size", (c.i64,) * 3, c.size_t)(M, K, R))


def pack8_da(du, p: Packed8, *, da=None, workspace=None, stream=None):
    """``dA = du.T @ x`` (fp32 [R, K]) of a packed ``x``: ``du`` [M, R] bf16. Bit for bit the dA of
    ``lora_delta_bwd`` for the unpacked x."""
    _is_packed(p, "p")
    M, R = du.shape
    K = p.cols
    c.check(du, "du", (M, R), torch.bfloat16)
    check_packed(p, "p", M, K, du.device)
    handle, on = c.run_on(stream)
    with on:
        da = torch.empty((R, K), dtype=torch.float32, device=du.device) if da is None else da
        if workspace is None:
            workspace = torch.empty(pack8_da_workspace_size(M, K, R), dtype=torch.uint8, device=du.device)
    c.check(da, "da", (R, K), torch.float32, device=du.device)
    c.done(c.fn("lora_pack8_da", _DA)(du.data_ptr(), p.codes.data_ptr(), p.scales.data_ptr(), M, K, R, da.data_ptr(),
                                      *c.scratch(workspace, du.device), handle), "lora_pack8_da")
    return da


def lora_delta_bwd_packed8_workspace_size(M: int, K: int, N: int, R: int) -> int:
    return int(c.fn("lora_delta_bwd_packed8_workspace_size", (c.i64,) * 4, c.size_t)(M, K, N, R))


def lora_delta_bwd_packed8(dy, p: Packed8, a, b, u, alpha: float, *, dx=None, da=None, db=None, du=None,
                           workspace=None, stream=None):
    """``lora_delta.lora_delta_bwd(dy, x, a, b, u, alpha)`` with x given as its 8-bit checkpoint:
    ``(dx, da, db, du)``, bit for bit those of the unpacked x. ``workspace`` (optional):
    ``lora_delta.new_workspace`` of the size above."""
    _is_packed(p, "p")
    M, N = dy.shape
    K, R = p.cols, a.shape[0]
    dev = dy.device
    c.check(dy, "dy", (M, N), torch.bfloat16)
    check_packed(p, "p", M, K, dev)
    c.check(a, "a", (R, K), torch.bfloat16, device=dev)
    c.check(b, "b", (N, R), torch.bfloat16, device=dev)
    c.check(u, "u", (M, R), torch.bfloat16, device=dev)
    handle, on = c.run_on(stream)
    with on:
        dx = torch.empty((M, K), dtype=torch.float32, device=dev) if dx is None else dx
        da = torch.empty((R, K), dtype=torch.float32, device=dev) if da is None else da
        db = torch.empty((N, R), dtype=torch.float32, device=dev) if db is None else db
        du = torch.empty((M, R), dtype=torch.bfloat16, device=dev) if du is None else du
        if workspace is None:
            workspace = _ld.new_workspace(lora_delta_bwd_packed8_workspace_size(M, K, N, R), dev)
    c.check(dx, "dx", (M, K), torch.float32, device=dev)
    c.check(da, "da", (R, K), torch.float32, device=dev)
    c.check(db, "db", (N, R), torch.float32, device=dev)
    c.check(du, "du", (M, R), torch.bfloat16, device=dev)
    c.done(c.fn("lora_delta_bwd_packed8", _BWD)(
        dy.data_ptr(), p.codes.data_ptr(), p.scales.data_ptr(), a.data_ptr(), b.data_ptr(), u.data_ptr(), float(alpha),
        M, K, N, R, dx.data_ptr(), da.data_ptr(), db.data_ptr(), du.data_ptr(), *c.scratch(workspace, dev), handle),
        "lora_delta_bwd_packed8")
    return dx, da, db, du
