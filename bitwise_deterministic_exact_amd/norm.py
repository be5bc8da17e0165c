"""Layer norm with its backward pass, for the layers around DetLinear.

  h = (x - mean) / sqrt(var + eps),  y = h * weight + bias     over the last dim
  g = dy * weight,  dx = rstd * (g - mean(g) - h * mean(g h))
  dweight = sum over rows of dy h,   dbias = sum over rows of dy

A row's results are a function of that row: not of how many rows there are,
nor of their strides or alignment.  The weights' gradients are sums over rows
(tokens): chunks of consecutive rows in float32 in one fixed order, the chunks
added exactly in the long accumulator and rounded once.  So rows sharded at
multiples of NORM_SHARD_ROWS (64) give, through layer_norm_digits,
det_combine and det_finalize, the bits of one call's float32 gradients over
all of them, as the K-shards of an exact GEMM do (det-train page, "Method").

x, the weights and y may each be float32 or bfloat16: a DetLinear's float32
output can be normalised straight into the bfloat16 input of the next one.
Arguments are checked in the compiled layer (csrc/head_ops.cpp): ValueError
for a bad shape, dtype or device.
Tracing a call (torch.jit.trace, make_fx) and forward-mode inputs are a
RuntimeError.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _lib

NORM_SHARD_ROWS = _lib.NORM_SHARD_ROWS
_DTYPES = (torch.float32, torch.bfloat16)


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out_dtype: Optional[torch.dtype] = None):
    """(y, mean, rstd): y of x's shape and ``out_dtype`` (default: x's),
    mean and rstd float32, one per row, for layer_norm_backward."""
    return _lib.ops().layer_norm_forward(x, weight, bias, eps, out_dtype)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, *, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True, grad_dtype: Optional[torch.dtype] = None,
                        digits: bool = False):
    """(dx, dweight, dbias) for the incoming gradient dy, each None when not
    needed; dx has x's dtype, the weights' gradients ``grad_dtype`` (default:
    weight's, or float32).  With ``digits`` a fourth value: the raw digits of
    dweight and dbias, int64 [2, C, 18], for det_combine."""
    r = _lib.ops().layer_norm_backward(dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias, grad_dtype,
                                       digits)
    return r if digits else r[:3]


def layer_norm_digits(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor) -> torch.Tensor:
    """Raw digits (int64 [2, C, 18]) of dweight and dbias over these rows.
    Row shards cut at multiples of NORM_SHARD_ROWS add with det_combine;
    det_finalize of the sum gives layer_norm_backward's float32 dweight and
    dbias over all rows, bit for bit."""
    return layer_norm_backward(dy, x, None, mean, rstd, need_dx=False, need_dweight=False, need_dbias=False,
                               digits=True)[3]


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Layer norm of x over its last dimension, differentiable (once, in
    reverse mode); see the module docstring.  x: float32 or bfloat16 [..., C], C <= 32768; weight and
    bias (both optional): [C], one dtype; result of ``out_dtype`` (default x's)."""
    return _lib.ops().layer_norm(x, weight, bias, eps, out_dtype)


class DetLayerNorm(torch.nn.Module):
    """Layer norm over the last dimension with learned weight (ones at the
    start) and bias (zeros); ``out_dtype`` as for layer_norm."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=torch.float32,
                 out_dtype: Optional[torch.dtype] = None):
        super().__init__()
        if not 1 <= features <= _lib.NORM_C_MAX:
            raise ValueError(f"features must lie in 1..{_lib.NORM_C_MAX}")
        if dtype not in _DTYPES or (out_dtype is not None and out_dtype not in _DTYPES):
            raise ValueError("DetLayerNorm supports float32 and bfloat16")
        if not 0.0 <= eps < math.inf:
            raise ValueError("eps must be >= 0 and finite")
        self.features, self.eps, self.out_dtype = features, eps, out_dtype
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return layer_norm(x, self.weight, self.bias, self.eps, self.out_dtype)

    def extra_repr(self) -> str:
        return f"features={self.features}, eps={self.eps}, bias={self.bias is not None}"
