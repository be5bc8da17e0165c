"""Losses of post-training on the log probabilities that token_logprobs forms:
the clipped policy loss with a KL term, and the preference loss over pairs of
answers, each with its gradient.

Per token of sampled answers, d = logprob - old_logprob, r = e^d, A its
advantage, q = ref_logprob - logprob:
  l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_weight k
  k = e^q - 1 - q
Per pair, s the sum over an answer's tokens of logprob - ref_logprob and
z = beta (s_chosen - s_rejected) - margin:
  sigmoid  -(1 - label_smoothing) ln sigma(z) - label_smoothing ln sigma(-z)
  hinge    max(0, 1 - z)
  ipo      (s_chosen - s_rejected - 1 / (2 beta))^2

A row's sums are formed in 64 bits in an order that its length alone decides;
the policy loss adds the rows' values exactly, divides in 64 bits and rounds once
(det-train page, "Method"), so it does not depend on the order of the rows.  exact_mean averages
a batch's preference losses the same way.

Tokens that a mask leaves out are not looked at, whatever they hold, and have no
gradient.  Arguments are checked in the compiled layer (csrc/policy_ops.cpp):
ValueError for a bad shape, dtype, device or value.  Tracing a call
(torch.jit.trace, make_fx) and forward-mode inputs are a RuntimeError.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib


class PolicyLoss(NamedTuple):
    """policy_loss' results, float32: the loss, and without a gradient the KL
    term's estimate k and the clipped tokens, reduced as the loss is (with
    "none": per token, clipped 0 or 1)."""
    loss: torch.Tensor
    kl: torch.Tensor
    clipped: torch.Tensor


class PreferenceLoss(NamedTuple):
    """preference_loss' results per pair, float32: the loss, and without a
    gradient the rewards beta * s of both answers."""
    loss: torch.Tensor
    chosen_reward: torch.Tensor
    rejected_reward: torch.Tensor


def policy_loss_forward(logprob: torch.Tensor, old_logprob: torch.Tensor, advantage: torch.Tensor,
                        mask: Optional[torch.Tensor] = None, *, ref_logprob: Optional[torch.Tensor] = None,
                        clip_low: float = 0.2, clip_high: float = 0.2, kl_weight: float = 0.0,
                        reduction: str = "tokens"):
    """(PolicyLoss, count): policy_loss without a graph, and the tokens that
    count (int64, one per row and the divisor; None with "none") for
    policy_loss_backward."""
    r = _lib.ops().policy_loss_forward(logprob, old_logprob, advantage, mask, ref_logprob, clip_low, clip_high,
                                       kl_weight, reduction)
    return PolicyLoss(*r[:3]), r[3]


def policy_loss_backward(g: torch.Tensor, logprob: torch.Tensor, old_logprob: torch.Tensor, advantage: torch.Tensor,
                         mask: Optional[torch.Tensor], count: Optional[torch.Tensor], *,
                         ref_logprob: Optional[torch.Tensor] = None, clip_low: float = 0.2, clip_high: float = 0.2,
                         kl_weight: float = 0.0, reduction: str = "tokens") -> torch.Tensor:
    """logprob's gradient for the incoming gradient g of the loss (float32 of its
    shape); ``count`` comes from policy_loss_forward."""
    return _lib.ops().policy_loss_backward(g, logprob, old_logprob, advantage, mask, ref_logprob, count, clip_low,
                                           clip_high, kl_weight, reduction)


def policy_loss(logprob: torch.Tensor, old_logprob: torch.Tensor, advantage: torch.Tensor,
                mask: Optional[torch.Tensor] = None, *, ref_logprob: Optional[torch.Tensor] = None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_weight: float = 0.0,
                reduction: str = "tokens") -> PolicyLoss:
    """The clipped policy loss; differentiable (once, in reverse mode) in
    ``logprob``, the other inputs are constants.

    logprob, old_logprob, ref_logprob: float32 [..., T], one row per answer;
    advantage: float32 [..., T] or one to a row [...]; mask: bool [..., T], False
    for tokens that do not count; clip_low in [0, 1], clip_high and kl_weight in
    [0, 1e6) (without a weight the KL estimate is only reported); reduction:
    "tokens", the mean over all tokens that count, "sequences", the mean of the
    rows' means (rows without a token left out), or "none", [..., T].  Nothing
    that counts: 0, and no gradient."""
    return PolicyLoss(*_lib.ops().policy_loss(logprob, old_logprob, advantage, mask, ref_logprob, clip_low, clip_high,
                                              kl_weight, reduction))


def preference_loss_forward(chosen_logprob: torch.Tensor, rejected_logprob: torch.Tensor,
                            ref_chosen_logprob: Optional[torch.Tensor] = None,
                            ref_rejected_logprob: Optional[torch.Tensor] = None, *,
                            chosen_mask: Optional[torch.Tensor] = None, rejected_mask: Optional[torch.Tensor] = None,
                            kind: str = "sigmoid", beta: float = 0.1, margin: float = 0.0,
                            label_smoothing: float = 0.0, by_length: bool = False):
    """(PreferenceLoss, slope): preference_loss without a graph, and the
    derivatives (float32 [pairs, 2]) for preference_loss_backward."""
    r = _lib.ops().preference_loss_forward(chosen_logprob, rejected_logprob, ref_chosen_logprob, ref_rejected_logprob,
                                           chosen_mask, rejected_mask, kind, beta, margin, label_smoothing, by_length)
    return PreferenceLoss(*r[:3]), r[3]


def preference_loss_backward(g: torch.Tensor, slope: torch.Tensor, chosen_shape, rejected_shape, *,
                             chosen_mask: Optional[torch.Tensor] = None,
                             rejected_mask: Optional[torch.Tensor] = None):
    """(dchosen, drejected) of the two shapes for the incoming gradient g (one
    per pair); ``slope`` comes from preference_loss_forward."""
    return _lib.ops().preference_loss_backward(g, slope, list(chosen_shape), list(rejected_shape), chosen_mask,
                                               rejected_mask)


def preference_loss(chosen_logprob: torch.Tensor, rejected_logprob: torch.Tensor,
                    ref_chosen_logprob: Optional[torch.Tensor] = None,
                    ref_rejected_logprob: Optional[torch.Tensor] = None, *,
                    chosen_mask: Optional[torch.Tensor] = None, rejected_mask: Optional[torch.Tensor] = None,
                    kind: str = "sigmoid", beta: float = 0.1, margin: float = 0.0, label_smoothing: float = 0.0,
                    by_length: bool = False) -> PreferenceLoss:
    """The preference loss of each pair; differentiable (once, in reverse mode)
    in both answers' log probabilities, the reference's are constants.

    chosen_logprob: float32 [..., Tc], rejected_logprob: float32 [..., Tr]; the
    reference's of the same shapes, both or neither; masks: bool, False for
    tokens that do not count; kind: "sigmoid", "hinge" or "ipo"; beta in
    (0, 1e6); margin finite (not with ipo); label_smoothing in [0, 0.5] (sigmoid
    only); by_length: means over the tokens in place of sums.  An answer
    without a token has the sum 0."""
    return PreferenceLoss(*_lib.ops().preference_loss(chosen_logprob, rejected_logprob, ref_chosen_logprob,
                                                      ref_rejected_logprob, chosen_mask, rejected_mask, kind, beta,
                                                      margin, label_smoothing, by_length))
