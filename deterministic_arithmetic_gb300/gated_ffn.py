"""The gated feed-forward block, forward and backward (``lora_gated_ffn_*`` of ``include/lora_mlp.h``).

``gated_ffn_fwd(x, w_gate, w_up)`` returns ``(h, gate, up)``, h = act(x w_gate.T) * (x w_up.T), both
projections, the activation and the product in one kernel; the LoRA deltas of the two projections
enter inside the activation (``delta_gate``, ``delta_up``: the outputs of ``lora_delta_fwd``).
``gated_ffn_bwd`` returns ``(dx, dgate, dup, dw_gate, dw_up)``; ``dgate`` and ``dup`` are also the
``dy`` of the two deltas' backward passes. There is no fallback.
"""
from __future__ import annotations

import torch

from . import _capi as c
from .pack8 import Packed8, check_packed, new_packed

ACTIVATIONS = {"silu": 0, "gelu": 1}
KEPT = {None: 0, "bf16": 1, "packed8": 2}

_FWD = (c.vp,) * 5 + (c.cint,) + (c.i64,) * 3 + (c.vp, c.cint) + (c.vp,) * 5
_BWD = (c.vp,) * 4 + (c.cint,) + (c.vp,) * 4 + (c.cint,) + (c.i64,) * 3 + (c.vp,) * 6


def _code(table: dict, key, name: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: expected one of {', '.join(map(repr, table))}, got {key!r}") from None


def _kept(t, name: str, M: int, F: int, device):
    """(address, scales' address) of a kept gate or up."""
    if isinstance(t, Packed8):
        check_packed(t, name, M, F, device)
        return t.codes.data_ptr(), t.scales.data_ptr()
    c.check(t, name, (M, F), torch.bfloat16, device=device)
    return t.data_ptr(), None


def gated_ffn_fwd(x, w_gate, w_up, *, activation: str = "silu", delta_gate=None, delta_up=None, save=None, h=None,
                  gate=None, up=None, stream=None):
    """``h = act(g) * u`` [M, F] bf16 with ``g = x @ w_gate.T + delta_gate``, ``u = x @ w_up.T + delta_up``.

    ``x`` [M, K], ``w_gate``, ``w_up`` [F, K] bf16 (K, F multiples of 8); the deltas fp32 [M, F], both
    or neither; ``activation`` "silu" or "gelu" (its tanh form). ``save`` keeps g and u for the
    backward pass: None (then ``gate`` and ``up`` come back as None), "bf16" or "packed8" (as
    ``Packed8``, rounded from fp32)."""
    M, K = x.shape
    F = w_gate.shape[0]
    dev = x.device
    act, keep = _code(ACTIVATIONS, activation, "activation"), _code(KEPT, save, "save")
    c.check(x, "x", (M, K), torch.bfloat16)
    c.check(w_gate, "w_gate", (F, K), torch.bfloat16, device=dev)
    c.check(w_up, "w_up", (F, K), torch.bfloat16, device=dev)
    if (delta_gate is None) != (delta_up is None):
        raise ValueError("delta_gate, delta_up: both or neither")
    if delta_gate is not None:
        c.check(delta_gate, "delta_gate", (M, F), torch.float32, device=dev)
        c.check(delta_up, "delta_up", (M, F), torch.float32, device=dev)
    handle, on = c.run_on(stream)
    with on:
        h = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if h is None else h
        if keep == 1:
            gate = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if gate is None else gate
            up = torch.empty((M, F), dtype=torch.bfloat16, device=dev) if up is None else up
        elif keep == 2:
            gate = new_packed(M, F, dev) if gate is None else gate
            up = new_packed(M, F, dev) if up is None else up
        else:
            gate = up = None
    c.check(h, "h", (M, F), torch.bfloat16, device=dev)
    gp = up_p = gs = us = None
    if keep:
        if isinstance(gate, Packed8) != (keep == 2) or isinstance(up, Packed8) != (keep == 2):
            raise ValueError(f"gate, up: expected {'Packed8' if keep == 2 else 'bf16 tensors'} for save={save!r}")
        (gp, gs), (up_p, us) = _kept(gate, "gate", M, F, dev), _kept(up, "up", M, F, dev)
    c.done(c.fn("lora_gated_ffn_fwd", _FWD)(
        x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), None if delta_gate is None else delta_gate.data_ptr(),
        None if delta_up is None else delta_up.data_ptr(), act, M, K, F, h.data_ptr(), keep, gp, up_p, gs, us, handle),
        "lora_gated_ffn_fwd")
    return h, gate, up


def gated_ffn_bwd(dh, x, w_gate, w_up, gate, up, *, activation: str = "silu", weight_grads: bool = True, dx=None,
                  dgate=None, dup=None, dw_gate=None, dw_up=None, stream=None):
    """``(dx, dgate, dup, dw_gate, dw_up)``, all bf16, of ``dh`` [M, F] bf16.

    ``gate`` and ``up`` are what the forward kept (both bf16 or both ``Packed8``). ``dup = dh act(g)``,
    ``dgate = dh u act'(g)``, rounded to bf16 and used so in ``dx = dgate @ w_gate + dup @ w_up`` and the
    weights' gradients ``dgate.T @ x``, ``dup.T @ x`` (None without ``weight_grads``: frozen weights;
    ``x`` may then be None)."""
    M, F = dh.shape
    K = w_gate.shape[1]
    dev = dh.device
    act = _code(ACTIVATIONS, activation, "activation")
    c.check(dh, "dh", (M, F), torch.bfloat16)
    if weight_grads or x is not None:
        c.check(x, "x", (M, K), torch.bfloat16, device=dev)
    c.check(w_gate, "w_gate", (F, K), torch.bfloat16, device=dev)
    c.check(w_up, "w_up", (F, K), torch.bfloat16, device=dev)
    if isinstance(gate, Packed8) != isinstance(up, Packed8):
        raise ValueError("gate, up: both bf16 tensors or both Packed8")
    (gp, gs), (up_p, us) = _kept(gate, "gate", M, F, dev), _kept(up, "up", M, F, dev)

    def out(t, *shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev) if t is None else t

    handle, on = c.run_on(stream)
    with on:
        dx, dgate, dup = out(dx, M, K), out(dgate, M, F), out(dup, M, F)
        if weight_grads:
            dw_gate, dw_up = out(dw_gate, F, K), out(dw_up, F, K)
        else:
            dw_gate = dw_up = None
    c.check(dx, "dx", (M, K), torch.bfloat16, device=dev)
    c.check(dgate, "dgate", (M, F), torch.bfloat16, device=dev)
    c.check(dup, "dup", (M, F), torch.bfloat16, device=dev)
    if weight_grads:
        c.check(dw_gate, "dw_gate", (F, K), torch.bfloat16, device=dev)
        c.check(dw_up, "dw_up", (F, K), torch.bfloat16, device=dev)
    c.done(c.fn("lora_gated_ffn_bwd", _BWD)(
        dh.data_ptr(), None if x is None else x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), 1 if gs is None else 2,
        gp, up_p, gs, us, act, M, K, F, dx.data_ptr(), dgate.data_ptr(), dup.data_ptr(),
        dw_gate.data_ptr() if weight_grads else None, dw_up.data_ptr() if weight_grads else None, handle),
        "lora_gated_ffn_bwd")
    return dx, dgate, dup, dw_gate, dw_up
