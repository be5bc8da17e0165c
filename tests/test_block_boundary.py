"""Refusals of the gated projection and the 8-bit checkpoints, on the CPU: the
C entry points reject bad arguments before any HIP call, and the Python layer
before any launch; and what torch's transforms may not do with them."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fw
from torch.fx.experimental.proxy_tensor import make_fx

import bitwise_deterministic_exact_amd as det
from bitwise_deterministic_exact_amd import _lib

P = ctypes.c_void_p
A, B = P(1 << 20), P(1 << 21)                       # never dereferenced: every case is refused
NULL, ODD = P(None), P((1 << 20) + 1)
EINVAL, EDTYPE = _lib.DET_EINVAL, _lib.DET_EDTYPE


def _gated(x=A, s_x=64, wg=A, s_g=64, wu=A, s_u=64, N=4, C=64, F=8, act=0, dt=1, h=B, save=0, gate=None, up=None, ge=None,
           ue=None, ws=B, n=1 << 30):
    return _lib.load().det_gated_linear(x, s_x, wg, s_g, wu, s_u, N, C, F, act, dt, h, save, gate, up, ge, ue, ws, n, None)


def _grad(dt=1, dh=A, s_dh=8, x=A, s_x=64, xe=None, wg=A, s_g=64, wu=A, s_u=64, save=1, gate=A, up=A, ge=None, ue=None, N=4,
          C=64, F=8, act=0, dx=B, dwg=B, dwu=B, ws=B, n=1 << 30):
    return _lib.load().det_gated_linear_grad(dt, dh, s_dh, x, s_x, xe, wg, s_g, wu, s_u, save, gate, up, ge, ue, N, C, F, act,
                                             dx, dwg, dwu, ws, n, None)


def _pack(dt=0, x=A, s=8, N=2, C=8, codes=B, exps=B):
    return _lib.load().det_int8_pack(dt, x, s, N, C, codes, exps, None)


def _unpack(codes=A, s=8, exps=A, N=2, C=8, dt=0, y=B):
    return _lib.load().det_int8_unpack(codes, s, exps, N, C, dt, y, None)


@pytest.mark.parametrize("call,want", [
    (lambda: _gated(dt=2), EDTYPE), (lambda: _gated(act=3), EINVAL), (lambda: _gated(act=-1), EINVAL),
    (lambda: _gated(save=3), EINVAL), (lambda: _gated(N=-1), EINVAL), (lambda: _gated(C=0), EINVAL),
    (lambda: _gated(F=0), EINVAL), (lambda: _gated(C=65537), EINVAL), (lambda: _gated(F=65537), EINVAL),
    (lambda: _gated(N=(1 << 22) + 1), EINVAL), (lambda: _gated(x=NULL), EINVAL), (lambda: _gated(wg=NULL), EINVAL),
    (lambda: _gated(wu=NULL), EINVAL), (lambda: _gated(s_x=-64), EINVAL), (lambda: _gated(s_u=-1), EINVAL),
    (lambda: _gated(x=ODD), EINVAL), (lambda: _gated(wu=ODD), EINVAL), (lambda: _gated(h=NULL), EINVAL),
    (lambda: _gated(h=P((1 << 21) + 2), dt=0), EINVAL), (lambda: _gated(save=1, gate=B), EINVAL),
    (lambda: _gated(save=1, gate=B, up=ODD), EINVAL), (lambda: _gated(save=2, gate=B, up=B, ge=B), EINVAL),
    # an operand that needs a padded copy, and no room for it
    (lambda: _gated(N=100, C=65, s_x=65, s_g=65, s_u=65, ws=NULL, n=0), EINVAL),
    (lambda: _gated(N=100, s_x=65, n=8), EINVAL), (lambda: _gated(N=100, x=P((1 << 20) + 2), ws=NULL), EINVAL),
    (lambda: _gated(N=100, s_x=0, ws=P((1 << 21) + 16)), EINVAL),
    (lambda: _grad(dt=5), EDTYPE), (lambda: _grad(act=9), EINVAL), (lambda: _grad(save=0), EINVAL),
    (lambda: _grad(save=3), EINVAL), (lambda: _grad(dwu=None), EINVAL), (lambda: _grad(dwg=None), EINVAL),
    (lambda: _grad(dh=NULL), EINVAL), (lambda: _grad(gate=NULL), EINVAL), (lambda: _grad(up=NULL), EINVAL),
    (lambda: _grad(save=2, ge=A), EINVAL), (lambda: _grad(s_dh=-8), EINVAL), (lambda: _grad(dt=0, dh=P((1 << 20) + 2)), EINVAL),
    (lambda: _grad(gate=ODD), EINVAL), (lambda: _grad(dx=ODD), EINVAL), (lambda: _grad(dwg=ODD), EINVAL),
    (lambda: _grad(x=NULL), EINVAL), (lambda: _grad(x=ODD), EINVAL), (lambda: _grad(s_x=-1), EINVAL),
    (lambda: _grad(wg=NULL), EINVAL), (lambda: _grad(s_u=-64), EINVAL), (lambda: _grad(ws=NULL), EINVAL),
    (lambda: _grad(n=100), EINVAL), (lambda: _grad(ws=P((1 << 21) + 128)), EINVAL), (lambda: _grad(C=65537), EINVAL),
    (lambda: _pack(dt=2), EDTYPE), (lambda: _pack(N=-1), EINVAL), (lambda: _pack(C=0), EINVAL),
    (lambda: _pack(C=(1 << 24) + 1), EINVAL), (lambda: _pack(s=-8), EINVAL), (lambda: _pack(N=(1 << 31) + 1), EINVAL),
    (lambda: _pack(x=NULL), EINVAL), (lambda: _pack(codes=NULL), EINVAL), (lambda: _pack(exps=NULL), EINVAL),
    (lambda: _pack(x=P((1 << 20) + 2)), EINVAL), (lambda: _pack(N=1 << 31, C=1 << 24, s=1 << 24), EINVAL),
    (lambda: _unpack(dt=-1), EDTYPE), (lambda: _unpack(N=-1), EINVAL), (lambda: _unpack(s=-1), EINVAL),
    (lambda: _unpack(codes=NULL), EINVAL), (lambda: _unpack(exps=NULL), EINVAL), (lambda: _unpack(y=NULL), EINVAL),
    (lambda: _unpack(dt=1, y=ODD), EINVAL),
])
def test_c_entry_points_refuse(call, want):
    assert call() == want
    assert _lib.last_error()


def test_empty_problems_are_no_ops():
    assert _gated(N=0, x=NULL, h=NULL) == _lib.DET_OK
    assert _grad(N=0, dwg=None, dwu=None) == _lib.DET_OK
    assert _grad(dx=None, dwg=None, dwu=None, dh=NULL) == _lib.DET_OK
    assert _pack(N=0, x=NULL) == _lib.DET_OK and _unpack(N=0, y=NULL) == _lib.DET_OK


def test_workspace_sizes():
    lib = _lib.load()
    fwd, grad = lib.det_gated_linear_workspace_bytes, lib.det_gated_linear_grad_workspace_bytes
    # none where the operands lie as the copies want them, or for few tokens of which nothing is kept
    assert fwd(1000, 128, 96, 0, 1) == 0 and fwd(64, 100, 96, 0, 0) == 0
    # else three copies with rows of a multiple of 64
    assert fwd(65, 100, 96, 0, 1) == 65 * 128 * 2 + 2 * 96 * 128 * 2
    assert fwd(64, 100, 96, 1, 1) == 64 * 128 * 2 + 2 * 96 * 128 * 2
    assert fwd(1000, 128, 96, 0, 0) == 1000 * 256 + 2 * 96 * 256
    # dg and du by token and by feature, x and the weights by feature
    assert grad(64, 128, 96, 1, 0) == 64 * 192 * 2 + 128 * 192 * 2
    assert grad(65, 128, 100, 0, 1) == 200 * 128 * 2 + 128 * 128 * 2
    assert grad(0, 128, 96, 1, 1) == 0 and fwd(10, 0, 8, 0, 0) == 0 and grad(10, 8, 1 << 17, 1, 1) == 0


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _i8(*shape):
    return _m(*shape, dtype=torch.int8)


S = det.GatedState(_m(2, 6), _m(2, 6))


@pytest.mark.parametrize("call,match", [
    (lambda: det.gated_linear(_m(2, 4, dtype=torch.float32), _m(6, 4), _m(6, 4)), "bfloat16"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4, dtype=torch.float32), _m(6, 4)), "w_gate"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4), _m(6, 5)), "w_up"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4), _m(7, 4)), "one shape"),
    (lambda: det.gated_linear(_m(2, 4), _m(4), _m(4)), "w_gate"),
    (lambda: det.gated_linear(_m(2, 0), _m(6, 0), _m(6, 0)), "at least 1"),
    (lambda: det.gated_linear(_m(), _m(6, 4), _m(6, 4)), "at least 1"),
    (lambda: det.gated_linear(_m(2, 4), _m(0, 4), _m(0, 4)), "w_gate"),
    (lambda: det.gated_linear(_m(2, 65537), _m(6, 65537), _m(6, 65537)), "65536"),
    (lambda: det.gated_linear(_m((1 << 22) + 1, 4), _m(6, 4), _m(6, 4)), "2\\^22"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4), _m(6, 4), activation="relu"), "activation"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4), _m(6, 4), checkpoint="fp8"), "checkpoint"),
    (lambda: det.gated_linear(_m(2, 4), _m(6, 4), _m(6, 4), out_dtype=torch.float16), "out_dtype"),
    (lambda: det.gated_linear(*(torch.zeros(s, dtype=torch.bfloat16) for s in ((2, 4), (6, 4), (6, 4)))), "GPU"),
    (lambda: det.gated_linear_backward(_m(2, 5), _m(2, 4), _m(6, 4), _m(6, 4), S), "dh"),
    (lambda: det.gated_linear_backward(_m(2, 6, dtype=torch.float16), _m(2, 4), _m(6, 4), _m(6, 4), S), "dh"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(_m(2, 6), _m(2, 5))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(_i8(2, 6), _i8(2, 6))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(
        det.PackedInt8(_i8(2, 6), _i8(2, 1)), _m(2, 6))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(
        det.PackedInt8(_i8(2, 6), _i8(2, 2)), det.PackedInt8(_i8(2, 6), _i8(2, 1)))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), det.PackedInt8(_i8(2, 4), _i8(2, 2)), _m(6, 4), _m(6, 4), S), "packed x"),
    (lambda: det.gated_linear_backward(_m(2, 6), det.PackedInt8(_m(2, 4), _i8(2, 1)), _m(6, 4), _m(6, 4), S), "packed x"),
    (lambda: det.DetGatedLinear(0, 4), "features"), (lambda: det.DetGatedLinear(4, 65537), "features"),
    (lambda: det.DetGatedLinear(4, 4, activation="tanh"), "activation"),
    (lambda: det.DetGatedLinear(4, 4, out_dtype=torch.float16), "out_dtype"),
    (lambda: det.DetGatedLinear(4, 4, checkpoint="int4"), "checkpoint"),
    (lambda: det.pack_int8(_m(2, 4, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: det.pack_int8(_m(2, 0)), "C"), (lambda: det.pack_int8(_m(1, (1 << 24) + 1)), "2\\^24"),
    (lambda: det.pack_int8(torch.zeros(2, 4)), "GPU"),
    (lambda: det.unpack_int8(det.PackedInt8(_i8(2, 40), _i8(2, 1))), "exponent"),
    (lambda: det.unpack_int8(det.PackedInt8(_i8(2, 40), _m(2, 2))), "int8"),
    (lambda: det.unpack_int8(det.PackedInt8(_i8(2, 40), _i8(2, 2)), torch.float16), "dtype"),
    (lambda: det.unpack_int8(det.PackedInt8(torch.zeros(2, 4, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.int8))), "GPU"),
])
def test_python_layer_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


@pytest.mark.parametrize("i", range(3))
@pytest.mark.parametrize("checkpoint", [None, "int8"])
def test_forward_mode_is_refused(i, checkpoint):
    args = [_m(2, 4), _m(6, 4), _m(6, 4)]
    with fw.dual_level():
        args[i] = fw.make_dual(args[i], _m(*args[i].shape))
        with pytest.raises(RuntimeError, match="forward-mode"):
            det.gated_linear(*args, checkpoint=checkpoint)


def test_traces_are_refused():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    x = z(2, 4)
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
    for call in (lambda x: det.gated_linear(x, z(6, 4), z(6, 4)), lambda x: det.gated_linear_forward(x, z(6, 4), z(6, 4))[0],
                 lambda x: det.gated_linear_backward(z(2, 6), x, z(6, 4), z(6, 4), det.GatedState(z(2, 6), z(2, 6)))[0],
                 lambda x: det.pack_int8(x)[0], lambda x: det.unpack_int8(det.PackedInt8(i8(2, 4), i8(2, 1))) + x):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(call, (x,), check_trace=False)
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(call)(x)


def test_gated_module():
    m = det.DetGatedLinear(6, 10, activation="gelu", checkpoint="int8")
    assert m.w_gate.shape == m.w_up.shape == (10, 6) and m.w_gate.dtype == torch.bfloat16
    assert not torch.equal(m.w_gate, m.w_up) and m.w_up.abs().max() <= 6 ** -0.5
    assert "gelu" in repr(m) and "int8" in repr(m)
