"""Activations kept in 8 bits between the forward and the backward pass.

Blocks of 32 consecutive elements of a row (the last may be shorter) share a
power of two 2^e; an element is code * 2^e with an int8 code.  e is the least
exponent with the block's largest magnitude below 127.5 * 2^e, in [-126, 121];
codes are rounded to nearest, ties to even, within +-127.  So a value is off by
at most half a unit, at most 1/127 of the block's largest, and what is read back
is exact in bfloat16 and float32: the exact products of DetLinear take it
without another rounding.

8.25 bits an element.  gated_linear and DetLinear keep what their backward pass
reads again this way with ``checkpoint="int8"``.

A block with a NaN or an infinity reads back as NaN throughout and sets
"nonfinite" in device_status().
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib


class PackedInt8(NamedTuple):
    """pack_int8's result: int8 codes [..., C] and one int8 exponent for each 32
    of them [..., ceil(C / 32)] (-128: a block that was not finite)."""
    codes: torch.Tensor
    exponents: torch.Tensor


def pack_int8(x: torch.Tensor) -> PackedInt8:
    """x (float32 or bfloat16 [..., C] on a GPU) in blocks of 8 bits; not
    differentiable: the gradient of what is kept is the layer's."""
    return PackedInt8(*_lib.ops().pack_int8(x.detach()))


def unpack_int8(packed: PackedInt8, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values that ``packed`` stands for, exactly, as float32 or bfloat16."""
    return _lib.ops().unpack_int8(packed[0], packed[1], dtype)
