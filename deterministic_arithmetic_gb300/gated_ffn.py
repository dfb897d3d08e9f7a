"""The gated feed-forward block, forward and backward (``lora_gated_ffn_*`` of ``include/lora_mlp.h``).

``gated_ffn_fwd(x, w_gate, w_up)`` returns ``(h, gate, up)``, h = act(x w_gate.T) * (x w_up.T), both
projections, the activation and the product in one kernel; the LoRA deltas of the two projections
enter inside the activation (``delta_gate``, ``delta_up``: the outputs of ``lora_delta_fwd``).
``gated_ffn_bwd`` returns ``(dx, dgate, dup, dw_gate, dw_up)``; ``dgate`` and ``dup`` are also the
``dy`` of the two deltas' backward passes. Every call takes ``stream=`` (default: the current stream).
No autograd graph records them. There is no fallback.
"""
from __future__ import annotations

from . import _capi as c

ACTIVATIONS = {"silu": 0, "gelu": 1}
KEPT = {None: 0, "bf16": 1, "packed8": 2}


def _code(table: dict, key, name: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name}: expected one of {', '.join(map(repr, table))}, got {key!r}") from None


@c.on_stream
def gated_ffn_fwd(x, w_gate, w_up, *, activation: str = "silu", delta_gate=None, delta_up=None, save=None, h=None,
                  gate=None, up=None):
    """``h = act(g) * u`` [M, F] bf16 with ``g = x @ w_gate.T + delta_gate``, ``u = x @ w_up.T + delta_up``.

    ``x`` [M, K], ``w_gate``, ``w_up`` [F, K] bf16 (K, F multiples of 8); the deltas fp32 [M, F], both
    or neither; ``activation`` "silu" or "gelu" (its tanh form). ``save`` keeps g and u for the
    backward pass: None (then ``gate`` and ``up`` come back as None), "bf16" or "packed8" (as
    ``Packed8``, rounded from fp32)."""
    act, keep = _code(ACTIVATIONS, activation, "activation"), _code(KEPT, save, "save")
    return c.mlp.gated_ffn_fwd(x, w_gate, w_up, act, delta_gate, delta_up, keep, h, gate, up)


@c.on_stream
def gated_ffn_bwd(dh, x, w_gate, w_up, gate, up, *, activation: str = "silu", weight_grads: bool = True, dx=None,
                  dgate=None, dup=None, dw_gate=None, dw_up=None):
    """``(dx, dgate, dup, dw_gate, dw_up)``, all bf16, of ``dh`` [M, F] bf16.

    ``gate`` and ``up`` are what the forward kept (both bf16 or both ``Packed8``). ``dup = dh act(g)``,
    ``dgate = dh u act'(g)``, rounded to bf16 and used so in ``dx = dgate @ w_gate + dup @ w_up`` and the
    weights' gradients ``dgate.T @ x``, ``dup.T @ x`` (None without ``weight_grads``: frozen weights;
    ``x`` may then be None)."""
    act = _code(ACTIVATIONS, activation, "activation")
    return c.mlp.gated_ffn_bwd(dh, x, w_gate, w_up, gate, up, act, weight_grads, dx, dgate, dup, dw_gate, dw_up)
