"""What a language model's head is trained and read with: the log
probabilities of given tokens, with entropy and top alternatives, and the
distillation loss against a teacher's top logits; each with its gradient.

For logits z of V tokens, scale s = 1 / temperature:
  l_j = s z_j - ln sum_i exp(s z_i),  p_j = exp(l_j)
  logprob = l_target,  entropy = -sum_j p_j l_j,  alternatives: the largest l_j
  distill = T^2 sum_k q_k (ln q_k - l_{index_k}),  q = softmax(teacher / T)

One pass reads the logits once; the gradients read them once more and write
theirs.  A row's results are a function of that row alone: the same bits in a
batch of one or of thousands, at any stride or alignment.

Masked tokens are -inf logits.  A row of nothing but -inf has log
probabilities -inf, entropy 0 and no gradient.  A row with a NaN or +inf has
NaN results (indices -1) and sets "nonfinite" in device_status().
Arguments are checked in the compiled layer (csrc/head_ops.cpp): ValueError
for a bad shape, dtype, device or value.
Tracing a call (torch.jit.trace, make_fx) and forward-mode inputs are a
RuntimeError.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib


class TokenLogProbs(NamedTuple):
    """token_logprobs' results: float32, int64 indices; logprob is None
    without targets."""
    logprob: Optional[torch.Tensor]
    entropy: torch.Tensor
    top_logprob: torch.Tensor
    top_index: torch.Tensor


def token_logprobs_forward(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                           top: int = 0, ignore_index: int = -100):
    """(TokenLogProbs, stat): the results without a graph, and the rows'
    float32 statistics [N, 4] for token_logprobs_backward."""
    r = _lib.ops().token_logprobs_forward(logits, targets, scale, top, ignore_index)
    return TokenLogProbs(*r[:4]), r[4]


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor], stat: torch.Tensor, *,
                            scale: float = 1.0, ignore_index: int = -100, top_index: Optional[torch.Tensor] = None,
                            g_logprob: Optional[torch.Tensor] = None, g_entropy: Optional[torch.Tensor] = None,
                            g_top: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The logits' gradient (their shape and dtype) for float32 incoming
    gradients of the log probability, the entropy and the alternatives, each
    optional; ``stat`` and ``top_index`` come from token_logprobs_forward."""
    return _lib.ops().token_logprobs_backward(logits, targets, stat, scale, ignore_index, top_index, g_logprob,
                                              g_entropy, g_top)


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                   top: int = 0, ignore_index: int = -100) -> TokenLogProbs:
    """Log probabilities of ``targets`` under softmax(scale * logits), the
    entropy, and the ``top`` most likely tokens with their log probabilities
    (ties to the lower index); differentiable (once, in reverse
    mode) in the logits.

    logits: float32 or bfloat16 [..., V]; targets: int64 [...] (None: no
    logprob), ``ignore_index`` gives 0 and no gradient, any other value outside
    [0, V) NaN and no gradient; top: 0..64.  Results are float32."""
    return TokenLogProbs(*_lib.ops().token_logprobs(logits, targets, scale, top, ignore_index))


def distill_forward(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_index: torch.Tensor, *,
                    temperature: float = 1.0):
    """(loss, stat, q): distill_loss without a graph, and what
    distill_backward needs (the rows' statistics and the teacher's
    probabilities, 0 in rows without a gradient)."""
    return _lib.ops().distill_forward(logits, teacher_logits, teacher_index, temperature)


def distill_backward(logits: torch.Tensor, teacher_index: torch.Tensor, stat: torch.Tensor, q: torch.Tensor,
                     g: torch.Tensor, *, temperature: float = 1.0) -> torch.Tensor:
    """The logits' gradient for the incoming gradient g of distill_loss;
    stat and q come from distill_forward."""
    return _lib.ops().distill_backward(logits, teacher_index, stat, q, g, temperature)


def distill_loss(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_index: torch.Tensor, *,
                 temperature: float = 1.0) -> torch.Tensor:
    """Per row T^2 KL(q || p): q the softmax of the teacher's K logits
    (renormalised over the K), p the student's over its whole vocabulary, both
    at temperature T; differentiable (once, in reverse mode) in the student's
    logits (the teacher is a constant).  float32 of the logits' leading shape; exact_mean
    gives the batch's mean.

    logits: float32 or bfloat16 [..., V]; teacher_logits: float32 or bfloat16
    [..., K], -inf for entries that are not there (their index is not looked
    at); teacher_index: int64 [..., K], an index may repeat; K <= 1024.  A row
    without any entry has the loss 0 and no gradient; one with an entry outside
    [0, V) the loss NaN and no gradient; a NaN or +inf among a row's teacher
    logits makes its loss and its whole gradient NaN."""
    return _lib.ops().distill_loss(logits, teacher_logits, teacher_index, temperature)
