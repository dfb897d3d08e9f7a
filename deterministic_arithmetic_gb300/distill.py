"""Distillation from a teacher's top logits, forward and backward (``lora_distill_topk_*`` of
``include/lora_base8.h``).

The loss of a row is the divergence of the student's distribution, softmax(logits / T) over the whole
vocabulary, from the teacher's, of which the largest logits and their ids are known: normalised over
themselves, or, with ``teacher_lse``, over the teacher's whole vocabulary, when the mass of what is not listed
is compared too. Logits are read once a pass. A row's results are the same bits in any batch. Every call takes
``stream=`` (default: the current stream). No autograd graph records them. There is no fallback.
"""
from __future__ import annotations

from . import _capi as c


@c.on_stream
def distill_topk_fwd(logits, ids, teacher, *, temperature: float = 1.0, teacher_lse=None, weight=None, loss=None,
                     probs=None, stats=None):
    """``(loss, probs, stats)`` of ``logits`` [M, V] (bf16 or fp32) against ``teacher`` [M, top] (bf16 or fp32), the
    teacher's logits at ``ids`` [M, top] (int64 or int32, top <= 1024).

    An id outside the vocabulary (-1, say), a logit of -infinity and a second entry of an id are no entries.
    ``teacher_lse`` [M] fp32: log(sum of exp(t / T)) over the teacher's vocabulary (``temperature`` counts with its 64 bits). ``weight`` [M] fp32 multiplies
    the loss; rows of weight 0 are not read. ``loss`` [M] is fp32, unreduced, without a factor of T * T; ``probs``
    [M, top] (the teacher's probabilities, -1 for no entry) and ``stats`` [M, 4] are for the backward pass. (New ones of up
    to 1 MiB together lie in one allocation.)"""
    return c.mlp.distill_topk_fwd(logits, ids, teacher, temperature, teacher_lse, weight, loss, probs, stats)


@c.on_stream
def distill_topk_bwd(dloss, logits, ids, probs, stats, *, temperature: float = 1.0, block8: bool = False,
                     dlogits=None):
    """The gradient by ``logits``, of their type, or, with ``block8``, as a ``Block8`` rounded from fp32: the ``dy`` of
    ``block8_linear_bwd``. ``dloss`` [M] fp32; ``probs`` and ``stats`` the forward's, ``ids`` and ``temperature`` as
    there. ``dlogits`` may be ``logits`` itself (which then holds the gradient)."""
    return c.mlp.distill_topk_bwd(dloss, logits, ids, probs, stats, temperature, block8, dlogits)
