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
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _DT, _call, _stream
from .norm import _ptr, _rows


class TokenLogProbs(NamedTuple):
    """token_logprobs' results: float32, int64 indices."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    top_logprob: torch.Tensor
    top_index: torch.Tensor


def _check_logits(logits, what: str):
    if not isinstance(logits, torch.Tensor):
        raise TypeError(f"{what}: logits must be a tensor")
    if logits.dtype not in _DT:
        raise ValueError(f"{what}: logits must be float32 or bfloat16 (got {logits.dtype})")
    if logits.dim() < 1 or not 1 <= logits.shape[-1] <= _lib.HEAD_V_MAX:
        raise ValueError(f"{what}: logits must be [..., V] with 1 <= V <= 2^24 (got shape {tuple(logits.shape)})")
    if logits.numel() // logits.shape[-1] > _lib.ROWS_MAX:
        raise ValueError(f"{what}: more than 2^22 rows in one call")


def _check_scale(scale: float, what: str) -> float:
    scale = float(scale)
    if not 1e-6 <= scale < 1e6:
        raise ValueError(f"{what}: the scale (1 / temperature) must lie in [1e-6, 1e6) (got {scale})")
    return scale


def _check_index(t, shape, device, name: str, what: str):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int64 or t.shape != shape or t.device != device:
        raise ValueError(f"{what}: {name} must be int64 of shape {tuple(shape)} on the logits' device")


def _on_gpu(t, what: str):
    if t.device.type != "cuda":
        raise ValueError(f"{what}: logits must be on a GPU")


def _grad_rows(g: Optional[torch.Tensor], shape):
    """An incoming gradient as (tensor, stride) over the flattened rows: a
    broadcast one stays one value."""
    if g is None:
        return None, 0
    if g.shape != shape or g.dtype != torch.float32:
        raise ValueError(f"incoming gradients must be float32 of shape {tuple(shape)}")
    if g.dim() == 1:
        return g, g.stride(0)
    if all(st == 0 or n == 1 for n, st in zip(g.shape, g.stride())):
        return g, 0
    return g.contiguous(), 1


def _workspace(N: int, V: int, top: int, device):
    nbytes = _lib.load().det_head_workspace_bytes(N, V, top)
    return (torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes) if nbytes else (None, 0)


def token_logprobs_forward(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                           top: int = 0, ignore_index: int = -100):
    """(TokenLogProbs, stat): the results without a graph, and the rows'
    float32 statistics [N, 4] for token_logprobs_backward."""
    what = "token_logprobs"
    _check_logits(logits, what)
    scale = _check_scale(scale, what)
    lead, V = logits.shape[:-1], logits.shape[-1]
    if not 0 <= top <= min(_lib.TOP_MAX, V):
        raise ValueError(f"{what}: top must lie in 0..min({_lib.TOP_MAX}, V) (got {top})")
    if targets is not None:
        _check_index(targets, lead, logits.device, "targets", what)
    _on_gpu(logits, what)
    dev = logits.device
    z = _rows(logits)
    N = z.shape[0]
    t = targets.reshape(-1) if targets is not None else None
    f32 = dict(dtype=torch.float32, device=dev)
    logprob = torch.empty(lead, **f32) if t is not None else None
    entropy = torch.empty(lead, **f32)
    stat = torch.empty((N, 4), **f32)
    top_logprob = torch.empty((*lead, top), **f32)
    top_index = torch.empty((*lead, top), dtype=torch.int64, device=dev)
    ws, nbytes = _workspace(N, V, top, dev)
    _call(dev, _lib.load().det_token_logprobs, _DT[z.dtype], _ptr(z), z.stride(0), N, V, scale, _ptr(t),
          t.stride(0) if t is not None else 0, int(ignore_index), top, _ptr(logprob), _ptr(entropy), _ptr(stat),
          _ptr(top_index), _ptr(top_logprob), _ptr(ws), nbytes, _stream(dev))
    return TokenLogProbs(logprob, entropy, top_logprob, top_index), stat


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor], stat: torch.Tensor, *,
                            scale: float = 1.0, ignore_index: int = -100, top_index: Optional[torch.Tensor] = None,
                            g_logprob: Optional[torch.Tensor] = None, g_entropy: Optional[torch.Tensor] = None,
                            g_top: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The logits' gradient (their shape and dtype) for incoming gradients of
    the log probability, the entropy and the alternatives, each optional;
    ``stat`` and ``top_index`` come from token_logprobs_forward."""
    what = "token_logprobs_backward"
    _check_logits(logits, what)
    scale = _check_scale(scale, what)
    lead, V = logits.shape[:-1], logits.shape[-1]
    z = _rows(logits)
    N = z.shape[0]
    if targets is not None:
        _check_index(targets, lead, logits.device, "targets", what)
    elif g_logprob is not None:
        raise ValueError(f"{what}: a gradient of the log probability needs the targets")
    if stat.shape != (N, 4) or stat.dtype != torch.float32 or stat.device != logits.device:
        raise ValueError(f"{what}: stat must be float32 [{N}, 4] on the logits' device")
    top = 0
    if g_top is not None:
        if top_index is None:
            raise ValueError(f"{what}: a gradient of the alternatives needs top_index")
        top = top_index.shape[-1]
        _check_index(top_index, torch.Size((*lead, top)), logits.device, "top_index", what)
        if g_top.shape != top_index.shape or g_top.dtype != torch.float32:
            raise ValueError(f"{what}: g_top must be float32 of top_index's shape")
        if top == 0:
            g_top = None
    _on_gpu(logits, what)
    dev = logits.device
    for g in (g_logprob, g_entropy, g_top):
        if g is not None and g.device != dev:
            raise ValueError(f"{what}: incoming gradients must be on the logits' device")
    t = targets.reshape(-1) if targets is not None else None
    glp, s_glp = _grad_rows(g_logprob, lead)
    gent, s_gent = _grad_rows(g_entropy, lead)
    gt = g_top.reshape(-1, top) if g_top is not None else None
    ti = top_index.reshape(-1, top).contiguous() if g_top is not None else None
    dz = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    _call(dev, _lib.load().det_token_logprobs_grad, _DT[z.dtype], _ptr(z), z.stride(0), N, V, scale, _ptr(t),
          t.stride(0) if t is not None else 0, int(ignore_index), top, _ptr(ti), _ptr(stat.contiguous()), _ptr(glp),
          s_glp, _ptr(gent), s_gent, _ptr(gt), gt.stride(0) if gt is not None else 0,
          gt.stride(1) if gt is not None else 0, _ptr(dz), V, _stream(dev))
    return dz


class _TokenLogProbsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale, top, ignore_index):
        out, stat = token_logprobs_forward(logits, targets, scale=scale, top=top, ignore_index=ignore_index)
        ctx.save_for_backward(logits, targets, stat, out.top_index if top else None)
        ctx.scale, ctx.ignore_index = scale, ignore_index
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(out.top_index)
        return tuple(out)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logprob, g_entropy, g_top, _):
        logits, targets, stat, top_index = ctx.saved_tensors
        if g_logprob is None and g_entropy is None and (g_top is None or top_index is None):
            return None, None, None, None, None
        dz = token_logprobs_backward(logits, targets, stat, scale=ctx.scale, ignore_index=ctx.ignore_index,
                                     top_index=top_index, g_logprob=g_logprob, g_entropy=g_entropy,
                                     g_top=g_top if top_index is not None else None)
        return dz, None, None, None, None


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                   top: int = 0, ignore_index: int = -100) -> TokenLogProbs:
    """Log probabilities of ``targets`` under softmax(scale * logits), the
    entropy, and the ``top`` most likely tokens with their log probabilities
    (ties to the lower index); differentiable in the logits.

    logits: float32 or bfloat16 [..., V]; targets: int64 [...] (None: no
    logprob), ``ignore_index`` gives 0 and no gradient, any other value outside
    [0, V) NaN and no gradient; top: 0..64.  Results are float32."""
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        return TokenLogProbs(*_TokenLogProbsFn.apply(logits, targets, scale, top, ignore_index))
    return token_logprobs_forward(logits, targets, scale=scale, top=top, ignore_index=ignore_index)[0]


def _check_teacher(logits, teacher, index, what: str):
    lead = logits.shape[:-1]
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in _DT or teacher.device != logits.device:
        raise ValueError(f"{what}: teacher logits must be float32 or bfloat16 on the logits' device")
    if teacher.dim() != len(lead) + 1 or teacher.shape[:-1] != lead or not 1 <= teacher.shape[-1] <= _lib.ENTRIES_MAX:
        raise ValueError(f"{what}: teacher logits must be [..., K] with the logits' leading shape and "
                         f"1 <= K <= {_lib.ENTRIES_MAX} (got {tuple(teacher.shape)})")
    _check_index(index, teacher.shape, logits.device, "the teacher's indices", what)


def distill_forward(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_index: torch.Tensor, *,
                    temperature: float = 1.0):
    """(loss, stat, q): distill_loss without a graph, and what
    distill_backward needs (the rows' statistics and the teacher's
    probabilities)."""
    what = "distill_loss"
    _check_logits(logits, what)
    temperature = float(temperature)
    if not temperature > 0.0:
        raise ValueError(f"{what}: the temperature must be positive (got {temperature})")
    _check_scale(1.0 / temperature, what)
    _check_teacher(logits, teacher_logits, teacher_index, what)
    _on_gpu(logits, what)
    dev = logits.device
    z, t, i = _rows(logits), _rows(teacher_logits), _rows(teacher_index)
    N, V = z.shape
    K = t.shape[1]
    f32 = dict(dtype=torch.float32, device=dev)
    loss = torch.empty(logits.shape[:-1], **f32)
    stat, q = torch.empty((N, 4), **f32), torch.empty((N, K), **f32)
    ws, nbytes = _workspace(N, V, 0, dev)
    _call(dev, _lib.load().det_distill, _DT[z.dtype], _ptr(z), z.stride(0), N, V, temperature, _DT[t.dtype], _ptr(t),
          t.stride(0), _ptr(i), i.stride(0), K, _ptr(loss), _ptr(stat), _ptr(q), _ptr(ws), nbytes, _stream(dev))
    return loss, stat, q


def distill_backward(logits: torch.Tensor, teacher_index: torch.Tensor, stat: torch.Tensor, q: torch.Tensor,
                     g: torch.Tensor, *, temperature: float = 1.0) -> torch.Tensor:
    """The logits' gradient for the incoming gradient g of distill_loss;
    stat and q come from distill_forward."""
    what = "distill_backward"
    _check_logits(logits, what)
    temperature = float(temperature)
    if not temperature > 0.0:
        raise ValueError(f"{what}: the temperature must be positive (got {temperature})")
    _check_scale(1.0 / temperature, what)
    z = _rows(logits)
    N, V = z.shape
    K = q.shape[-1]
    if q.shape != (N, K) or q.dtype != torch.float32 or stat.shape != (N, 4) or stat.dtype != torch.float32:
        raise ValueError(f"{what}: stat must be float32 [{N}, 4] and q float32 [{N}, K]")
    if not 1 <= K <= _lib.ENTRIES_MAX:
        raise ValueError(f"{what}: K must lie in 1..{_lib.ENTRIES_MAX}")
    _check_index(teacher_index, torch.Size((*logits.shape[:-1], K)), logits.device, "the teacher's indices", what)
    _on_gpu(logits, what)
    dev = logits.device
    if any(v.device != dev for v in (stat, q, g)):
        raise ValueError(f"{what}: stat, q and g must be on the logits' device")
    i = _rows(teacher_index)
    gv, s_g = _grad_rows(g, logits.shape[:-1])
    dz = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    _call(dev, _lib.load().det_distill_grad, _DT[z.dtype], _ptr(z), z.stride(0), N, V, temperature, _ptr(i),
          i.stride(0), K, _ptr(stat.contiguous()), _ptr(q.contiguous()), _ptr(gv), s_g, _ptr(dz), V, _stream(dev))
    return dz


class _DistillFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_logits, teacher_index, temperature):
        loss, stat, q = distill_forward(logits, teacher_logits, teacher_index, temperature=temperature)
        ctx.save_for_backward(logits, teacher_index, stat, q)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        logits, teacher_index, stat, q = ctx.saved_tensors
        return distill_backward(logits, teacher_index, stat, q, g, temperature=ctx.temperature), None, None, None


def distill_loss(logits: torch.Tensor, teacher_logits: torch.Tensor, teacher_index: torch.Tensor, *,
                 temperature: float = 1.0) -> torch.Tensor:
    """Per row T^2 KL(q || p): q the softmax of the teacher's K logits
    (renormalised over the K), p the student's over its whole vocabulary, both
    at temperature T; differentiable in the student's logits (the teacher is a
    constant).  float32 of the logits' leading shape; exact_mean gives the
    batch's mean.

    logits: float32 or bfloat16 [..., V]; teacher_logits: float32 or bfloat16
    [..., K], -inf for entries that are not there (their index is not looked
    at); teacher_index: int64 [..., K], an index may repeat; K <= 1024.  A row
    without any entry has the loss 0 and no gradient."""
    if isinstance(teacher_logits, torch.Tensor):
        teacher_logits = teacher_logits.detach()
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        return _DistillFn.apply(logits, teacher_logits, teacher_index, temperature)
    return distill_forward(logits, teacher_logits, teacher_index, temperature=temperature)[0]
