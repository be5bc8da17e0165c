"""The gated projection between a norm and a DetLinear, with its backward pass.

  g = x w_gate^T,  u = x w_up^T,  h = act(g) * u
  dg = dh u act'(g),  du = dh act(g)
  dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x

One kernel forms both products, the activation and their product on the matrix
cores, for one token as for thousands.  Sums are float32 in one fixed order: a
token's h and dx are the same bits in any batch, layout or launch (the sums are
not exact as DetLinear's are; a weight gradient is a sum over the call's rows in
their order).  h is rounded once; the gradients round dg and du to bfloat16 for
the matrix cores and each sum once.

The backward pass reads x and both projections again; these are kept as fp16
elements of blocks of 32 that share a power of two (11 bits each, no overflow).
With ``checkpoint="int8"`` x and both projections are kept in 8 bits
(packed.py), half the bytes: the result h is the same, the gradients are those
at the values that the 8 bits stand for.

Arguments are checked in the compiled layer (csrc/block_ops.cpp): ValueError for
a bad shape, dtype, device or value.  Tracing a call (torch.jit.trace, make_fx)
and forward-mode inputs are a RuntimeError.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from .packed import PackedInt8


class ScaledHalf(NamedTuple):
    """fp16 values [..., F] and one int8 exponent e for each 32 of them [...,
    ceil(F / 32)]: an element is value * 2^e."""
    values: torch.Tensor
    exponents: torch.Tensor


class GatedState(NamedTuple):
    """What gated_linear_backward reads again: both projections of the forward
    pass, as ScaledHalf or (checkpoint "int8") PackedInt8."""
    gate: Union[ScaledHalf, PackedInt8]
    up: Union[ScaledHalf, PackedInt8]


def gated_linear_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, activation: str = "silu",
                         out_dtype: Optional[torch.dtype] = None, checkpoint: Optional[str] = None):
    """(h, GatedState): gated_linear without a graph, and what
    gated_linear_backward needs besides x and the weights."""
    h, gate, up, ge, ue = _lib.ops().gated_linear_forward(x, w_gate, w_up, activation, out_dtype, checkpoint)
    kind = PackedInt8 if checkpoint == "int8" else ScaledHalf
    return h, GatedState(kind(gate, ge), kind(up, ue))


def gated_linear_backward(dh: torch.Tensor, x: Union[torch.Tensor, PackedInt8, None], w_gate: torch.Tensor,
                          w_up: torch.Tensor, state: GatedState, *, activation: str = "silu", need_dx: bool = True,
                          need_dw: bool = True):
    """(dx, dw_gate, dw_up), bfloat16, each None when not needed, for the
    incoming gradient dh of h (float32 or bfloat16).  x as the forward pass had
    it, or pack_int8 of it (None without need_dw); ``state`` comes from
    gated_linear_forward."""
    x, xe = x if isinstance(x, PackedInt8) else (x, None)
    (gate, ge), (up, ue) = state
    return _lib.ops().gated_linear_backward(dh, x, xe, w_gate, w_up, gate, up, ge, ue, activation, need_dx, need_dw)


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, activation: str = "silu",
                 out_dtype: Optional[torch.dtype] = None, checkpoint: Optional[str] = None) -> torch.Tensor:
    """act(x w_gate^T) * (x w_up^T), differentiable (once, in reverse mode); see
    the module docstring.

    x: bfloat16 [..., C]; w_gate, w_up: bfloat16 [F, C]; C, F <= 65536;
    activation: "silu", "gelu" (exact) or "gelu_tanh"; result [..., F] of
    ``out_dtype`` (bfloat16, the default, or float32); checkpoint: None or "int8"."""
    return _lib.ops().gated_linear(x, w_gate, w_up, activation, out_dtype, checkpoint)


class DetGatedLinear(torch.nn.Module):
    """gated_linear with learned bfloat16 weights [hidden_features,
    in_features]; a DetLinear(hidden_features, in_features) after it completes
    a feed-forward block.  Unlike DetLinear's its sums are float32: repeatable, a
    token's the same in any batch, but the weights' gradients depend on how the
    rows are cut into calls."""

    def __init__(self, in_features: int, hidden_features: int, activation: str = "silu", device=None,
                 out_dtype: Optional[torch.dtype] = None, checkpoint: Optional[str] = None):
        super().__init__()
        if not (1 <= in_features <= _lib.GATED_MAX and 1 <= hidden_features <= _lib.GATED_MAX):
            raise ValueError(f"features must lie in 1..{_lib.GATED_MAX}")
        if activation not in ("silu", "gelu", "gelu_tanh"):
            raise ValueError('activation must be "silu", "gelu" or "gelu_tanh"')
        if out_dtype not in (None, torch.float32, torch.bfloat16):
            raise ValueError("out_dtype must be float32 or bfloat16")
        if checkpoint not in (None, "int8"):
            raise ValueError('checkpoint must be None or "int8"')
        self.in_features, self.hidden_features = in_features, hidden_features
        self.activation, self.out_dtype, self.checkpoint = activation, out_dtype, checkpoint
        bound = 1.0 / math.sqrt(in_features)
        for name in ("w_gate", "w_up"):
            w = torch.empty(hidden_features, in_features, dtype=torch.float32).uniform_(-bound, bound)
            setattr(self, name, torch.nn.Parameter(w.to(device=device, dtype=torch.bfloat16)))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return gated_linear(x, self.w_gate, self.w_up, activation=self.activation, out_dtype=self.out_dtype,
                            checkpoint=self.checkpoint)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, hidden_features={self.hidden_features}, "
                f"activation={self.activation}" + (f", checkpoint={self.checkpoint}" if self.checkpoint else ""))
