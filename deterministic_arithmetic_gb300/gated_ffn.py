"""The gated feed-forward block, forward and backward (``lora_gated_ffn_*`` of ``include/lora_mlp.h``).

``gated_ffn_fwd(x, w_gate, w_up)`` returns ``(h, gate, up)``, h = act(x w_gate.T) * (x w_up.T), both
projections, the activation and the product in one kernel; the LoRA deltas of the two projections
enter inside the activation (``delta_gate``, ``delta_up``: the outputs of ``lora_delta_fwd``).
``gated_ffn_bwd`` returns ``(dx, dgate, dup, dw_gate, dw_up)``; ``dgate`` and ``dup`` are also the
``dy`` of the two deltas' backward passes. Every call takes ``stream=`` (default: the current stream).
There is no fallback.
"""
from __future__ import annotations

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


def _kept(t, name: str, M: int, F: int, device: int):
    """(address, scales' address) of a kept gate or up."""
    if isinstance(t, Packed8):
        return check_packed(t, name, M, F, device)
    return c.check(t, name, (M, F), c.BF16, device), None


@c.on_stream
def gated_ffn_fwd(x, w_gate, w_up, *, activation: str = "silu", delta_gate=None, delta_up=None, save=None, h=None,
                  gate=None, up=None):
    """``h = act(g) * u`` [M, F] bf16 with ``g = x @ w_gate.T + delta_gate``, ``u = x @ w_up.T + delta_up``.

    ``x`` [M, K], ``w_gate``, ``w_up`` [F, K] bf16 (K, F multiples of 8); the deltas fp32 [M, F], both
    or neither; ``activation`` "silu" or "gelu" (its tanh form). ``save`` keeps g and u for the
    backward pass: None (then ``gate`` and ``up`` come back as None), "bf16" or "packed8" (as
    ``Packed8``, rounded from fp32)."""
    dev = c.device_of(x, "x")
    M, K = x.shape
    F = w_gate.shape[0]
    act, keep = _code(ACTIVATIONS, activation, "activation"), _code(KEPT, save, "save")
    xp = c.check(x, "x", (M, K), c.BF16, dev)
    wgp, wup = c.check(w_gate, "w_gate", (F, K), c.BF16, dev), c.check(w_up, "w_up", (F, K), c.BF16, dev)
    dgp = dup = None
    if delta_gate is not None or delta_up is not None:
        dgp = c.check(delta_gate, "delta_gate", (M, F), c.F32, dev)      # both or neither
        dup = c.check(delta_up, "delta_up", (M, F), c.F32, dev)
    h = c.out(h, "h", (M, F), c.BF16, dev)
    gp = up_p = gs = us = None
    if keep == 0:
        gate = up = None
    else:
        if gate is None:
            gate = new_packed(M, F, dev) if keep == 2 else c.empty((M, F), dtype=c.BF16, device=dev)
        if up is None:
            up = new_packed(M, F, dev) if keep == 2 else c.empty((M, F), dtype=c.BF16, device=dev)
        if isinstance(gate, Packed8) != (keep == 2) or isinstance(up, Packed8) != (keep == 2):
            raise ValueError(f"gate, up: expected {'Packed8' if keep == 2 else 'bf16 tensors'} for save={save!r}")
        (gp, gs), (up_p, us) = _kept(gate, "gate", M, F, dev), _kept(up, "up", M, F, dev)
    c.done(c.fn("lora_gated_ffn_fwd", _FWD)(xp, wgp, wup, dgp, dup, act, M, K, F, h.data_ptr(), keep, gp, up_p, gs, us,
                                            c.stream(dev)), "lora_gated_ffn_fwd")
    return h, gate, up


@c.on_stream
def gated_ffn_bwd(dh, x, w_gate, w_up, gate, up, *, activation: str = "silu", weight_grads: bool = True, dx=None,
                  dgate=None, dup=None, dw_gate=None, dw_up=None):
    """``(dx, dgate, dup, dw_gate, dw_up)``, all bf16, of ``dh`` [M, F] bf16.

    ``gate`` and ``up`` are what the forward kept (both bf16 or both ``Packed8``). ``dup = dh act(g)``,
    ``dgate = dh u act'(g)``, rounded to bf16 and used so in ``dx = dgate @ w_gate + dup @ w_up`` and the
    weights' gradients ``dgate.T @ x``, ``dup.T @ x`` (None without ``weight_grads``: frozen weights;
    ``x`` may then be None)."""
    dev = c.device_of(dh, "dh")
    M, F = dh.shape
    K = w_gate.shape[1]
    act = _code(ACTIVATIONS, activation, "activation")
    dhp = c.check(dh, "dh", (M, F), c.BF16, dev)
    xp = c.check(x, "x", (M, K), c.BF16, dev) if weight_grads or x is not None else None
    wgp, wup = c.check(w_gate, "w_gate", (F, K), c.BF16, dev), c.check(w_up, "w_up", (F, K), c.BF16, dev)
    if isinstance(gate, Packed8) != isinstance(up, Packed8):
        raise ValueError("gate, up: both bf16 tensors or both Packed8")
    (gp, gs), (up_p, us) = _kept(gate, "gate", M, F, dev), _kept(up, "up", M, F, dev)
    dx = c.out(dx, "dx", (M, K), c.BF16, dev)
    dgate, dup = c.out(dgate, "dgate", (M, F), c.BF16, dev), c.out(dup, "dup", (M, F), c.BF16, dev)
    dwg = dwu = None
    if weight_grads:
        dw_gate, dw_up = c.out(dw_gate, "dw_gate", (F, K), c.BF16, dev), c.out(dw_up, "dw_up", (F, K), c.BF16, dev)
        dwg, dwu = dw_gate.data_ptr(), dw_up.data_ptr()
    else:
        dw_gate = dw_up = None
    c.done(c.fn("lora_gated_ffn_bwd", _BWD)(
        dhp, xp, wgp, wup, 1 if gs is None else 2, gp, up_p, gs, us, act, M, K, F, dx.data_ptr(), dgate.data_ptr(),
        dup.data_ptr(), dwg, dwu, c.stream(dev)), "lora_gated_ffn_bwd")
    return dx, dgate, dup, dw_gate, dw_up
