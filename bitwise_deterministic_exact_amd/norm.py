"""Layer norm with its backward pass, for the layers around DetLinear.

  h = (x - mean) / sqrt(var + eps),  y = h * weight + bias     over the last dim
  g = dy * weight,  dx = rstd * (g - mean(g) - h * mean(g h))
  dweight = sum over rows of dy h,   dbias = sum over rows of dy

A row's results are a function of that row: not of how many rows there are,
nor of their strides or alignment.  The weights' gradients are sums over rows
(tokens): chunks of consecutive rows in float32 in one fixed order, the chunks
added exactly in the long accumulator and rounded once.  So rows sharded at
multiples of NORM_SHARD_ROWS (32) give, through layer_norm_digits,
det_combine and det_finalize, the bits of one call over all of them, as the
K-shards of an exact GEMM do (det-train page, "Method").

x, the weights and y may each be float32 or bfloat16: a DetLinear's float32
output can be normalised straight into the bfloat16 input of the next one.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import _lib
from .api import _DT, _call, _stream

NORM_SHARD_ROWS = _lib.NORM_SHARD_ROWS


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _rows(t: torch.Tensor) -> torch.Tensor:
    """[..., C] as [N, C] with adjacent elements in a row (a copy only when
    the rows cannot be described by one stride, or their elements are apart)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    return t if t.shape[1] <= 1 or t.stride(1) == 1 else t.contiguous()


def _check(x, weight, bias, what: str) -> None:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what}: x must be a tensor")
    if x.dtype not in _DT:
        raise ValueError(f"{what}: x must be float32 or bfloat16 (got {x.dtype})")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{what}: x needs a last dimension of at least 1 (got shape {tuple(x.shape)})")
    if x.shape[-1] > _lib.NORM_C_MAX:
        raise ValueError(f"{what}: rows of {x.shape[-1]} exceed the limit {_lib.NORM_C_MAX}")
    if x.numel() // x.shape[-1] > _lib.ROWS_MAX:
        raise ValueError(f"{what}: more than 2^22 rows in one call")
    dt = None
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        if p.dtype not in _DT or p.shape != x.shape[-1:] or p.device != x.device:
            raise ValueError(f"{what}: {name} must be float32 or bfloat16 of shape [{x.shape[-1]}] on x's device")
        if dt is not None and p.dtype != dt:
            raise ValueError(f"{what}: weight and bias must share a dtype")
        dt = p.dtype
    if x.device.type != "cuda":
        raise ValueError(f"{what}: x must be on a GPU")


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       out_dtype: Optional[torch.dtype] = None):
    """(y, mean, rstd): y of x's shape and ``out_dtype`` (default: x's),
    mean and rstd float32, one per row, for layer_norm_backward."""
    _check(x, weight, bias, "layer_norm")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DT:
        raise ValueError(f"layer_norm: out_dtype must be float32 or bfloat16 (got {out_dtype})")
    if not 0.0 <= eps < 1e30:
        raise ValueError("layer_norm: eps must be >= 0 and finite")
    x2 = _rows(x)
    N, C = x2.shape
    y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    stat = torch.empty((2, N), dtype=torch.float32, device=x.device)
    mean, rstd = stat.unbind(0)
    w = weight.contiguous() if weight is not None else None
    b = bias.contiguous() if bias is not None else None
    wdt = _DT[w.dtype if w is not None else b.dtype if b is not None else torch.float32]
    _call(x.device, _lib.load().det_layer_norm, _DT[x.dtype], _ptr(x2), x2.stride(0), wdt, _ptr(w), _ptr(b), N, C,
          float(eps), _DT[out_dtype], _ptr(y), _ptr(mean), _ptr(rstd), _stream(x.device))
    return y, mean.reshape(x.shape[:-1]), rstd.reshape(x.shape[:-1])


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, *, need_dx: bool = True, need_dweight: bool = True,
                        need_dbias: bool = True, grad_dtype: Optional[torch.dtype] = None,
                        digits: bool = False):
    """(dx, dweight, dbias) for the incoming gradient dy, each None when not
    needed; dx has x's dtype, the weights' gradients ``grad_dtype`` (default:
    weight's, or float32).  With ``digits`` a fourth value: the raw digits of
    dweight and dbias, int64 [2, C, 18], for det_combine."""
    _check(x, weight, None, "layer_norm_backward")
    if dy.shape != x.shape or dy.dtype not in _DT or dy.device != x.device:
        raise ValueError("layer_norm_backward: dy must be float32 or bfloat16 of x's shape on x's device")
    for s in (mean, rstd):
        if s.dtype != torch.float32 or s.numel() != x.numel() // x.shape[-1] or s.device != x.device:
            raise ValueError("layer_norm_backward: mean and rstd must be float32, one per row, on x's device")
    if grad_dtype is None:
        grad_dtype = weight.dtype if weight is not None else torch.float32
    if grad_dtype not in _DT:
        raise ValueError("layer_norm_backward: grad_dtype must be float32 or bfloat16")
    x2, dy2 = _rows(x), _rows(dy)
    N, C = x2.shape
    dev = x.device
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_dx else None
    dw = torch.empty(C, dtype=grad_dtype, device=dev) if need_dweight else None
    db = torch.empty(C, dtype=grad_dtype, device=dev) if need_dbias else None
    dg = torch.empty((2, C, _lib.NUM_DIGITS), dtype=torch.int64, device=dev) if digits else None
    lib = _lib.load()
    ws, nbytes = None, 0
    if need_dweight or need_dbias or digits:
        nbytes = lib.det_layer_norm_grad_workspace_bytes(N, C)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    w = weight.contiguous() if weight is not None else None
    if w is not None and w.dtype != grad_dtype:
        w = w.to(grad_dtype) if grad_dtype == torch.float32 else w
        if w.dtype != grad_dtype:
            raise ValueError("layer_norm_backward: a float32 weight takes float32 gradients")
    _call(dev, lib.det_layer_norm_grad, _DT[x.dtype], _ptr(x2), x2.stride(0), _DT[dy.dtype], _ptr(dy2),
          dy2.stride(0), _DT[grad_dtype], _ptr(w), _ptr(mean.contiguous()), _ptr(rstd.contiguous()), N, C, _ptr(dx),
          _ptr(dw), _ptr(db), _ptr(dg), _ptr(ws), nbytes, _stream(dev))
    return (dx, dw, db, dg) if digits else (dx, dw, db)


def layer_norm_digits(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor) -> torch.Tensor:
    """Raw digits (int64 [2, C, 18]) of dweight and dbias over these rows.
    Row shards cut at multiples of NORM_SHARD_ROWS add with det_combine;
    det_finalize of the sum gives layer_norm_backward's float32 dweight and
    dbias over all rows, bit for bit."""
    return layer_norm_backward(dy, x, None, mean, rstd, need_dx=False, need_dweight=False, need_dbias=False,
                               digits=True)[3]


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = (weight if weight is not None else bias if bias is not None else mean).dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(dy, x, weight, mean, rstd, need_dx=need[0], need_dweight=need[1],
                                         need_dbias=need[2], grad_dtype=ctx.param_dtype)
        return dx, dw, db, None, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Layer norm of x over its last dimension, differentiable; see the module
    docstring.  x: float32 or bfloat16 [..., C], C <= 32768; weight and bias
    (both optional): [C], one dtype; result of ``out_dtype`` (default x's)."""
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, weight, bias)):
        return _LayerNormFn.apply(x, weight, bias, eps, out_dtype)
    return layer_norm_forward(x, weight, bias, eps, out_dtype)[0]


class DetLayerNorm(torch.nn.Module):
    """Layer norm over the last dimension with learned weight (ones at the
    start) and bias (zeros); ``out_dtype`` as for layer_norm."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=torch.float32,
                 out_dtype: Optional[torch.dtype] = None):
        super().__init__()
        if not 1 <= features <= _lib.NORM_C_MAX:
            raise ValueError(f"features must lie in 1..{_lib.NORM_C_MAX}")
        if dtype not in _DT or (out_dtype is not None and out_dtype not in _DT):
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
