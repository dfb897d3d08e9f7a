"""One training step of an adapter on a frozen layer, under a frozen head, both held in 8 bits; the loss compares the student's
distribution with the largest logits that a teacher gave:
    h = x W^T + delta(x);  n = layer norm of h;  logits = n H^T;  loss = distance from the teacher, a row each.

The weights take a byte each and serve both passes. The gradient by the logits leaves the loss in 8 bits, as the
products take it; a bf16 one is never written.

    python examples/distill_step.py [tokens] [width] [vocabulary] [rank]
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deterministic_arithmetic_gb300 import block8, distill, layer_norm, lora_delta  # noqa: E402


@dataclass
class Student:
    """Frozen: ``w`` and ``head`` in blocks of 128 x 128. Trained: the norm's parameters (fp32) and the adapter's ``a`` [R, K] and
    ``b`` [K, R] (bf16)."""
    w: block8.Block8
    head: block8.Block8
    ln_weight: torch.Tensor
    ln_bias: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    alpha: float = 2.0
    temperature: float = 2.0


@dataclass
class Teacher:
    """Its largest logits a row, their ids, and the log of the sum of exp(t / T) over its whole vocabulary; ``weight`` 0 takes
    a row (padding, say) out."""
    ids: torch.Tensor
    logits: torch.Tensor
    lse: torch.Tensor
    weight: torch.Tensor


def forward(p: Student, x, t: Teacher):
    """(the rows' losses, what the backward pass needs)."""
    delta, u = lora_delta.lora_delta_fwd(x, p.a, p.b, p.alpha)
    h = block8.block8_linear_fwd(block8.block8(x), p.w, delta=delta)
    n, mean, rstd = layer_norm.layer_norm_fwd(h, p.ln_weight, p.ln_bias)
    logits = block8.block8_linear_fwd(block8.block8(n), p.head)
    loss, probs, stats = distill.distill_topk_fwd(logits, t.ids, t.logits, temperature=p.temperature, teacher_lse=t.lse,
                                                  weight=t.weight)
    return loss, (x, u, h, mean, rstd, logits, probs, stats)


def backward(p: Student, t: Teacher, dloss, kept):
    """dx, and the gradients of what is trained."""
    x, u, h, mean, rstd, logits, probs, stats = kept
    dlogits = distill.distill_topk_bwd(dloss, logits, t.ids, probs, stats, temperature=p.temperature, block8=True)
    dn = block8.block8_linear_bwd(dlogits, p.head)
    dh, dw, db = layer_norm.layer_norm_bwd(dn, h, p.ln_weight, mean, rstd)
    dx_delta, da, db_, _ = lora_delta.lora_delta_bwd(dh, x, p.a, p.b, u, p.alpha)
    dx = block8.block8_linear_bwd(block8.block8(dh), p.w, delta=dx_delta)
    return dx, dict(ln_weight=dw, ln_bias=db, a=da, b=db_)


def make(tokens: int, width: int, vocabulary: int, rank: int, top: int = 64, seed: int = 0):
    """A student, its input and a teacher's answers, random; the last row in eight has weight 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, c=1.0, dtype=torch.bfloat16):
        return (torch.randn(*s, generator=g, device="cuda") * c).to(dtype)

    f32 = torch.float32
    p = Student(block8.block8(rnd(width, width, c=width ** -0.5), tile=128), block8.block8(rnd(vocabulary, width, c=width ** -0.5), tile=128),
                1 + rnd(width, c=0.1, dtype=f32), rnd(width, c=0.1, dtype=f32), rnd(rank, width, c=width ** -0.5), rnd(width, rank, c=rank ** -0.5))
    full = rnd(tokens, vocabulary, c=3.0)
    logits, ids = torch.topk(full, min(top, vocabulary), dim=1)
    lse = torch.logsumexp(full.float() / p.temperature, 1)
    weight = torch.ones(tokens, device="cuda")
    weight[7::8] = 0
    return p, rnd(tokens, width), Teacher(ids, logits, lse, weight)


def main() -> None:
    tokens, width, vocabulary, rank = (int(v) for v in (sys.argv[1:] + ["4096", "4096", "131072", "16"][len(sys.argv) - 1:]))
    p, x, t = make(tokens, width, vocabulary, rank)
    dloss = torch.full((tokens,), 1.0 / tokens, device="cuda")

    def step():
        loss, kept = forward(p, x, t)
        return loss, backward(p, t, dloss, kept)

    for _ in range(3):
        loss, (dx, grads) = step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        step()
    end.record()
    torch.cuda.synchronize()
    weights = sum(w.codes.nbytes + w.scales.nbytes for w in (p.w, p.head))
    print(f"{tokens} tokens, width {width}, vocabulary {vocabulary}, rank {rank}: {start.elapsed_time(end) / 10:.3f} ms a step; "
          f"weights {weights / 2 ** 20:.1f} MiB; mean loss {loss.mean().item():.4g}")
    for name, g in dict(dx=dx, **grads).items():
        print(f"  {name:10s} {tuple(g.shape)} norm {g.float().norm().item():.4g}")


if __name__ == "__main__":
    main()
