"""One training step of adapters on a frozen gated MLP, with everything the backward pass needs kept in
8 bits:  x -> layer norm -> n;  h = silu(n Wg^T + delta_g(n)) * (n Wu^T + delta_u(n)).

Kept between the passes: the packed x and n, the packed gate and up values, the norm's two statistics a
row and the adapters' U rows; x, n, gate and up in bf16 are not. The adapters' deltas enter inside the
activation, so the gated block's backward pass hands each adapter its dY.

    python examples/mlp_block_step.py [tokens] [width] [hidden] [rank]
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deterministic_arithmetic_gb300 import gated_ffn, layer_norm, lora_delta, pack8  # noqa: E402


@dataclass
class Block:
    """Frozen weights bf16, the norm's parameters fp32; the adapters (a [R, K], b [F, R] bf16) of the gate
    and up projections share ``alpha``."""
    ln_weight: torch.Tensor
    ln_bias: torch.Tensor
    w_gate: torch.Tensor
    w_up: torch.Tensor
    a_gate: torch.Tensor
    b_gate: torch.Tensor
    a_up: torch.Tensor
    b_up: torch.Tensor
    alpha: float = 2.0


def forward(p: Block, x):
    """(h, what the backward pass needs)."""
    n, mean, rstd = layer_norm.layer_norm_fwd(x, p.ln_weight, p.ln_bias)
    delta_gate, u_gate = lora_delta.lora_delta_fwd(n, p.a_gate, p.b_gate, p.alpha)
    delta_up, u_up = lora_delta.lora_delta_fwd(n, p.a_up, p.b_up, p.alpha)
    h, gate, up = gated_ffn.gated_ffn_fwd(n, p.w_gate, p.w_up, delta_gate=delta_gate, delta_up=delta_up, save="packed8")
    return h, (pack8.pack8(x), mean, rstd, pack8.pack8(n), gate, up, u_gate, u_up)


def backward(p: Block, dh, kept):
    """dx, and the gradients of everything that is trained."""
    x, mean, rstd, n, gate, up, u_gate, u_up = kept
    dn, dgate, dup, _, _ = gated_ffn.gated_ffn_bwd(dh, None, p.w_gate, p.w_up, gate, up, weight_grads=False)
    dn_gate, da_gate, db_gate, _ = pack8.lora_delta_bwd_packed8(dgate, n, p.a_gate, p.b_gate, u_gate, p.alpha)
    dn_up, da_up, db_up, _ = pack8.lora_delta_bwd_packed8(dup, n, p.a_up, p.b_up, u_up, p.alpha)
    dn = (dn_gate.add_(dn_up).add_(dn)).to(torch.bfloat16)
    dx, dw, db = layer_norm.layer_norm_bwd(dn, x, p.ln_weight, mean, rstd)
    return dx, dict(ln_weight=dw, ln_bias=db, a_gate=da_gate, b_gate=db_gate, a_up=da_up, b_up=db_up)


def make(tokens: int, width: int, hidden: int, rank: int, seed: int = 0):
    """A block, its input and the gradient of its output, random."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, c=1.0, dtype=torch.bfloat16):
        return (torch.randn(*s, generator=g, device="cuda") * c).to(dtype)

    f32 = torch.float32
    p = Block(1 + rnd(width, c=0.1, dtype=f32), rnd(width, c=0.1, dtype=f32), rnd(hidden, width, c=width ** -0.5),
              rnd(hidden, width, c=width ** -0.5), rnd(rank, width, c=width ** -0.5), rnd(hidden, rank, c=rank ** -0.5),
              rnd(rank, width, c=width ** -0.5), rnd(hidden, rank, c=rank ** -0.5))
    return p, rnd(tokens, width), rnd(tokens, hidden, c=0.1)


def main() -> None:
    tokens, width, hidden, rank = (int(v) for v in (sys.argv[1:] + ["4096", "5120", "17408", "16"][len(sys.argv) - 1:]))
    p, x, dh = make(tokens, width, hidden, rank)

    def step():
        h, kept = forward(p, x)
        return h, kept, backward(p, dh, kept)

    for _ in range(3):
        h, kept, (dx, grads) = step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    rows = sum(t.codes.nbytes + t.scales.nbytes for t in kept if isinstance(t, pack8.Packed8))
    print(f"{tokens} tokens, {width} -> {hidden}, rank {rank}: {start.elapsed_time(end) / 10:.3f} ms a step; kept in 8 "
          f"bits {rows / 2 ** 20:.1f} MiB (bf16: {2 * (2 * x.numel() + 2 * h.numel()) / 2 ** 20:.1f} MiB)")
    for name, g in dict(dx=dx, **grads).items():
        print(f"  {name:10s} {tuple(g.shape)} norm {g.float().norm().item():.4g}")


if __name__ == "__main__":
    main()
