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
           ue=None, ws=B, n=1 << 30, s_k=8):
    return _lib.load().det_gated_linear(x, s_x, wg, s_g, wu, s_u, N, C, F, act, dt, h, save, gate, up, s_k, ge, ue, ws, n, None)


def _grad(dt=1, dh=A, s_dh=8, x=A, s_x=64, xe=None, wg=A, s_g=64, wu=A, s_u=64, save=1, gate=A, up=A, ge=A, ue=A, N=4,
          C=64, F=8, act=0, dx=B, dwg=B, dwu=B, ws=B, n=1 << 30,
          s_k=8):
    return _lib.load().det_gated_linear_grad(dt, dh, s_dh, x, s_x, xe, wg, s_g, wu, s_u, save, gate, up, s_k, ge, ue, N, C, F, act,
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
    (lambda: _gated(h=P((1 << 21) + 2), dt=0), EINVAL), (lambda: _gated(save=1, gate=B), EINVAL), (lambda: _gated(save=1, gate=B, up=B, ge=B, ue=B, s_k=7), EINVAL),
    (lambda: _grad(s_k=-8), EINVAL), (lambda: _gated(save=1, gate=B, up=B, ge=B), EINVAL),
    (lambda: _gated(save=1, gate=B, up=ODD, ge=B, ue=B), EINVAL), (lambda: _gated(save=2, gate=B, up=B, ge=B), EINVAL),
    # an operand that needs a padded copy, and no room for it
    (lambda: _gated(N=100, C=65, s_x=65, s_g=65, s_u=65, ws=NULL, n=0), EINVAL),
    (lambda: _gated(N=100, s_x=65, n=8), EINVAL), (lambda: _gated(N=100, x=P((1 << 20) + 2), ws=NULL), EINVAL),
    (lambda: _gated(N=100, s_x=0, ws=P((1 << 21) + 16)), EINVAL),
    (lambda: _grad(dt=5), EDTYPE), (lambda: _grad(act=9), EINVAL), (lambda: _grad(save=0), EINVAL),
    (lambda: _grad(save=3), EINVAL), (lambda: _grad(dwu=None), EINVAL), (lambda: _grad(dwg=None), EINVAL),
    (lambda: _grad(dh=NULL), EINVAL), (lambda: _grad(gate=NULL), EINVAL), (lambda: _grad(up=NULL), EINVAL),
    (lambda: _grad(save=2, ue=None), EINVAL), (lambda: _grad(ge=None), EINVAL), (lambda: _grad(s_dh=-8), EINVAL), (lambda: _grad(dt=0, dh=P((1 << 20) + 2)), EINVAL),
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


def test_what_no_launch_could_hold_is_refused():
    for call in (lambda: _gated(N=1 << 22, F=4097), lambda: _gated(N=1 << 22, C=4160, s_x=4160, s_g=4160, s_u=4160),
                 lambda: _grad(N=1 << 22, F=4097, s_dh=4097, s_k=4128), lambda: _pack(N=(1 << 31) - 1, C=33, s=33),
                 lambda: _unpack(N=1 << 24, C=(1 << 12) + 1, s=4097), lambda: _policy(Bn=1 << 22, T=1025),
                 lambda: _policy_grad(Bn=1 << 12, T=(1 << 20) + 1), lambda: _prefer(Pn=1 << 22, Tr=1025),
                 lambda: _prefer_grad(Pn=1 << 22, Tc=1025)):
        assert call() == EINVAL and "in one call" in _lib.last_error()


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
    # dg and du with rows of a multiple of 64 each, copies where an operand does not lie as wanted, x where it is packed
    assert grad(64, 128, 96, 1, 1, 1, 0) == 64 * 2 * 128 * 2
    assert grad(64, 128, 96, 1, 1, 0, 0) == 64 * 2 * 128 * 2 + 2 * 96 * 256 + 64 * 256
    assert grad(65, 100, 128, 0, 1, 1, 0) == 65 * 2 * 128 * 2 + 65 * 128 * 2
    assert grad(64, 128, 96, 1, 1, 1, 1) == 64 * 2 * 128 * 2 + 64 * 256
    assert grad(0, 128, 96, 1, 1, 1, 0) == 0 and fwd(10, 0, 8, 0, 0) == 0 and grad(10, 8, 1 << 17, 1, 1, 1, 0) == 0
    assert grad(10, 8, 8, 0, 0, 0, 0) == 0


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _i8(*shape):
    return _m(*shape, dtype=torch.int8)


def _half(*shape):
    return det.ScaledHalf(_m(*shape, dtype=torch.float16), _i8(*shape[:-1], (shape[-1] + 31) // 32))


S = det.GatedState(_half(2, 6), _half(2, 6))


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
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(_half(2, 6), _half(2, 5))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(
        det.ScaledHalf(_m(2, 6), _i8(2, 1)), _half(2, 6))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(
        det.PackedInt8(_i8(2, 6), _i8(2, 1)), _half(2, 6))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6, 4), _m(6, 4), det.GatedState(
        det.PackedInt8(_i8(2, 6), _i8(2, 2)), det.PackedInt8(_i8(2, 6), _i8(2, 1)))), "gate and up"),
    (lambda: det.gated_linear_backward(_m(2, 6), det.PackedInt8(_i8(2, 4), _i8(2, 2)), _m(6, 4), _m(6, 4), S), "packed x"),
    (lambda: det.gated_linear_backward(_m(2, 6), det.PackedInt8(_m(2, 4), _i8(2, 1)), _m(6, 4), _m(6, 4), S), "packed x"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(3, 4), _m(6, 4), _m(6, 4), S), "x must be"),
    (lambda: det.gated_linear_backward(_m(2, 6), None, _m(6, 4), _m(6, 4), S), "need x"),
    (lambda: det.gated_linear_backward(_m(2, 6), _m(2, 4), _m(6), _m(6, 4), S), "w_gate"),
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
                 lambda x: det.gated_linear_backward(z(2, 6), x, z(6, 4), z(6, 4), det.GatedState(
                     *[det.ScaledHalf(z(2, 6).half(), i8(2, 1))] * 2))[0],
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


# ---------------------------------------------------------------- policy and preference losses

F64 = ctypes.c_double


def _policy(lp=A, old=A, adv=A, s=8, adv_t=1, mask=None, s_mask=8, ref=None, Bn=2, T=8, low=0.2, high=0.2, beta=0.0, red=1, loss=B,
            kl=B, clipped=B, count=B, ws=B, n=1 << 20):
    return _lib.load().det_policy_loss(lp, s, old, 8, adv, 8, adv_t, mask, s_mask, ref, 8, Bn, T, low, high, beta, red, loss, kl,
                                       clipped, count, ws, n, None)


def _policy_grad(lp=A, red=1, count=A, g=A, s_g=0, s_gt=0, d=B, Bn=2, T=8, low=0.2, ref=None, beta=0.0):
    return _lib.load().det_policy_loss_grad(lp, 8, A, 8, A, 8, 1, None, 0, ref, 8, Bn, T, low, 0.2, beta, red, count, g, s_g, s_gt,
                                            d, None)


def _prefer(c=A, r=A, rc=None, rr=None, s=8, Tc=8, Tr=8, Pn=2, kind=0, beta=0.1, margin=0.0, smooth=0.0, loss=B, rew=B, slope=B):
    return _lib.load().det_preference_loss(c, s, rc, 8, None, 0, Tc, r, 8, rr, 8, None, 0, Tr, Pn, kind, beta, margin, smooth, 0,
                                           loss, rew, B, slope, None)


def _prefer_grad(s_m=0, Tc=8, Tr=8, Pn=2, slope=A, g=A, s_g=1, dc=B, dr=B):
    return _lib.load().det_preference_loss_grad(None, s_m, Tc, None, 0, Tr, Pn, slope, g, s_g, dc, dr, None)


O2, O4, N8 = P((1 << 20) + 2), P((1 << 21) + 4), float("nan")


@pytest.mark.parametrize("call", [
    lambda: _policy(Bn=-1), lambda: _policy(T=-1), lambda: _policy(Bn=(1 << 22) + 1), lambda: _policy(T=(1 << 24) + 1),
    lambda: _policy(Bn=1 << 21, T=1 << 20), lambda: _policy(s=-1), lambda: _policy(s_mask=-8), lambda: _policy(low=-0.1),
    lambda: _policy(low=1.5), lambda: _policy(low=N8), lambda: _policy(high=-1.0), lambda: _policy(high=N8),
    lambda: _policy(high=1e6), lambda: _policy(beta=-1.0), lambda: _policy(beta=N8), lambda: _policy(beta=0.1),
    lambda: _policy(adv_t=2), lambda: _policy(red=3), lambda: _policy(red=-1), lambda: _policy(lp=NULL), lambda: _policy(old=NULL),
    lambda: _policy(adv=NULL), lambda: _policy(lp=O2), lambda: _policy(ref=O2), lambda: _policy(loss=NULL), lambda: _policy(kl=NULL),
    lambda: _policy(clipped=NULL), lambda: _policy(count=NULL), lambda: _policy(count=O4), lambda: _policy(loss=O2),
    lambda: _policy(ws=NULL), lambda: _policy(n=7), lambda: _policy(ws=P((1 << 21) + 8)),
    lambda: _policy_grad(lp=NULL), lambda: _policy_grad(red=7), lambda: _policy_grad(count=NULL), lambda: _policy_grad(g=NULL),
    lambda: _policy_grad(s_g=-1), lambda: _policy_grad(s_gt=-1), lambda: _policy_grad(d=NULL), lambda: _policy_grad(d=O2),
    lambda: _policy_grad(low=2.0), lambda: _policy_grad(beta=1.0), lambda: _policy_grad(count=O4),
    lambda: _prefer(Pn=-1), lambda: _prefer(Tc=-1), lambda: _prefer(Tr=-1), lambda: _prefer(Tr=(1 << 24) + 1), lambda: _prefer(s=-1),
    lambda: _prefer(kind=3), lambda: _prefer(beta=0.0), lambda: _prefer(beta=N8), lambda: _prefer(margin=N8),
    lambda: _prefer(margin=0.5, kind=2), lambda: _prefer(smooth=0.6), lambda: _prefer(smooth=-0.1), lambda: _prefer(smooth=0.1, kind=1),
    lambda: _prefer(rc=A), lambda: _prefer(rr=A), lambda: _prefer(c=NULL), lambda: _prefer(r=NULL), lambda: _prefer(loss=NULL),
    lambda: _prefer(rew=NULL), lambda: _prefer(slope=NULL), lambda: _prefer(c=O2), lambda: _prefer(slope=O2),
    lambda: _prefer_grad(Pn=-1), lambda: _prefer_grad(Tc=-1), lambda: _prefer_grad(s_m=-1), lambda: _prefer_grad(slope=NULL),
    lambda: _prefer_grad(g=NULL), lambda: _prefer_grad(s_g=-1), lambda: _prefer_grad(dc=O2), lambda: _prefer_grad(g=O2),
])
def test_loss_entry_points_refuse(call):
    assert call() == EINVAL and _lib.last_error()


def test_empty_losses_are_no_ops():
    assert _policy(Bn=0, red=0, lp=NULL, loss=NULL) == _lib.DET_OK and _policy(T=0, red=0, loss=NULL) == _lib.DET_OK
    assert _policy_grad(T=0, d=NULL) == _lib.DET_OK and _prefer(Pn=0, loss=NULL) == _lib.DET_OK
    assert _prefer_grad(dc=NULL, dr=NULL) == _lib.DET_OK and _prefer_grad(Tc=0, Tr=0) == _lib.DET_OK


def test_loss_workspace_sizes():
    f = _lib.load().det_policy_loss_workspace_bytes
    # per piece (2048 tokens, or a row of up to 512) two sums in 64 bits and two counts; per workgroup that joins rows 35 words
    assert f(3, 512, 1) == 3 * 24 + 35 * 8 and f(3, 513, 2) == 3 * 24 + 35 * 8 and f(3, 2049, 2) == 6 * 24 + 35 * 8
    assert f((1 << 13) + 1, 512, 1) == ((1 << 13) + 1) * 24 + 2 * 35 * 8
    assert f(3, 512, 0) == 0 and f(0, 512, 1) == 0 and f(3, 0, 1) == 0


def _f(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


M = lambda *s: _f(*s, dtype=torch.bool)


@pytest.mark.parametrize("call,match", [
    (lambda: det.policy_loss(_f(2, 4, dtype=torch.bfloat16), _f(2, 4), _f(2)), "float32"),
    (lambda: det.policy_loss(_f(), _f(), _f()), "logprob"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 5), _f(2)), "old_logprob"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(4)), "advantage"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, dtype=torch.float64)), "advantage"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), _f(2, 4)), "mask"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), M(2, 3)), "mask"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), ref_logprob=_f(4)), "ref_logprob"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), kl_weight=0.1), "ref_logprob"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), clip_low=1.1), "clip_low"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), clip_high=-0.1), "clip_high"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), ref_logprob=_f(2, 4), kl_weight=-1.0), "kl_weight"),
    (lambda: det.policy_loss(_f(2, 4), _f(2, 4), _f(2, 4), reduction="mean"), "reduction"),
    (lambda: det.policy_loss(torch.zeros(2, 4), torch.zeros(2, 4), torch.zeros(2)), "GPU"),
    (lambda: det.policy_loss_backward(_f(2), _f(2, 4), _f(2, 4), _f(2), None, None), "GPU|gradient"),
    (lambda: det.preference_loss(_f(2, 4, dtype=torch.bfloat16), _f(2, 4)), "chosen_logprob"),
    (lambda: det.preference_loss(_f(2, 4), _f()), "rejected_logprob"),
    (lambda: det.preference_loss(_f(2, 4), _f(3, 4)), "leading shape"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 4), _f(2, 4)), "both sides or for none"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), _f(2, 4), _f(2, 4)), "ref_rejected"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), chosen_mask=M(2, 5)), "chosen_mask"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), rejected_mask=_f(2, 5)), "rejected_mask"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), kind="dpo"), "kind"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), beta=0.0), "beta"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), margin=float("inf")), "margin"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), margin=1.0, kind="ipo"), "margin"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), label_smoothing=0.7), "label_smoothing"),
    (lambda: det.preference_loss(_f(2, 4), _f(2, 5), label_smoothing=0.1, kind="hinge"), "label_smoothing"),
    (lambda: det.preference_loss(torch.zeros(2, 4), torch.zeros(2, 4)), "GPU"),
    (lambda: det.preference_loss_backward(_f(2), _f(3, 2), (2, 4), (2, 5)), "slope"),
    (lambda: det.preference_loss_backward(_f(3), _f(2, 2), (2, 4), (2, 5)), "gradient"),
    (lambda: det.preference_loss_backward(_f(2), _f(2, 2), (2, 4), (3, 5)), "leading shape"),
    (lambda: det.DetLinear(4, 4, checkpoint="bf16"), "checkpoint"),
])
def test_loss_python_layer_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


@pytest.mark.parametrize("i", range(4))
def test_losses_refuse_forward_mode(i):
    args = [_f(2, 4) for _ in range(4)]
    with fw.dual_level():
        args[i] = fw.make_dual(args[i], _f(2, 4))
        with pytest.raises(RuntimeError, match="forward-mode"):
            det.policy_loss(*args[:3], ref_logprob=args[3])
        with pytest.raises(RuntimeError, match="forward-mode"):
            det.preference_loss(*args)


def test_losses_refuse_traces():
    z = torch.zeros
    x = z(2, 4)
    for call in (lambda x: det.policy_loss(x, z(2, 4), z(2)).loss, lambda x: det.policy_loss_forward(x, z(2, 4), z(2))[0].loss,
                 lambda x: det.policy_loss_backward(z(()), x, z(2, 4), z(2), None, z(3, dtype=torch.int64)),
                 lambda x: det.preference_loss(x, z(2, 5)).loss, lambda x: det.preference_loss_forward(x, z(2, 5))[1],
                 lambda x: det.preference_loss_backward(x[:, 0], z(2, 2), (2, 4), (2, 5))[0]):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(call, (x,), check_trace=False)
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(call)(x)
