"""Refusals of layer norm, token log probabilities and distillation, on the
CPU: the C entry points reject bad arguments before any HIP call, and the
Python layer before any launch."""
import ctypes

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from bitwise_deterministic_exact_amd import _lib

P = ctypes.c_void_p
A, B = P(1 << 20), P(1 << 21)                       # never dereferenced: every case is refused


def _norm(x_dt=0, x=A, s_x=8, w_dt=0, w=A, b=A, N=4, C=8, eps=1e-5, y_dt=0, y=B, mean=B, rstd=B):
    return _lib.load().det_layer_norm(x_dt, x, s_x, w_dt, w, b, N, C, eps, y_dt, y, mean, rstd, None)


def _norm_grad(x_dt=0, x=A, s_x=8, y_dt=0, dy=A, s_dy=8, w_dt=0, w=A, mean=A, rstd=A, N=4, C=8, dx=B, dw=B, db=B,
               digits=None, ws=B, n=1 << 20):
    return _lib.load().det_layer_norm_grad(x_dt, x, s_x, y_dt, dy, s_dy, w_dt, w, mean, rstd, N, C, dx, dw, db,
                                           digits, ws, n, None)


def _score(dt=0, z=A, s=8, N=2, V=8, scale=1.0, target=A, s_t=1, ignore=-100, top=2, lp=B, ent=B, stat=B, ti=B,
           tl=B, ws=B, n=1 << 20):
    return _lib.load().det_token_logprobs(dt, z, s, N, V, scale, target, s_t, ignore, top, lp, ent, stat, ti, tl, ws,
                                          n, None)


def _score_grad(dt=0, z=A, s=8, N=2, V=8, scale=1.0, target=A, s_t=1, top=0, ti=None, stat=A, glp=A, s_glp=1,
                gent=None, gtop=None, dz=B, s_dz=8):
    return _lib.load().det_token_logprobs_grad(dt, z, s, N, V, scale, target, s_t, -100, top, ti, stat, glp, s_glp,
                                               gent, 1, gtop, 1, 1, dz, s_dz, None)


def _distill(dt=0, z=A, N=2, V=8, T=1.0, tdt=0, t=A, s_t=3, i=A, s_i=3, K=3, loss=B, stat=B, q=B):
    return _lib.load().det_distill(dt, z, 8, N, V, T, tdt, t, s_t, i, s_i, K, loss, stat, q, B, 1 << 20, None)


def _distill_grad(T=1.0, i=A, K=3, stat=A, q=A, g=A, s_g=1, dz=B, s_dz=8):
    return _lib.load().det_distill_grad(0, A, 8, 2, 8, T, i, 3, K, stat, q, g, s_g, dz, s_dz, None)


EINVAL, EDTYPE = _lib.DET_EINVAL, _lib.DET_EDTYPE
NULL = P(None)


@pytest.mark.parametrize("call,want", [
    (lambda: _norm(x_dt=2), EDTYPE), (lambda: _norm(w_dt=-1), EDTYPE), (lambda: _norm(y_dt=7), EDTYPE),
    (lambda: _norm(N=-1), EINVAL), (lambda: _norm(C=0), EINVAL), (lambda: _norm(C=32769), EINVAL),
    (lambda: _norm(N=(1 << 22) + 1), EINVAL), (lambda: _norm(s_x=-1), EINVAL), (lambda: _norm(x=NULL), EINVAL),
    (lambda: _norm(y=NULL), EINVAL), (lambda: _norm(x=P((1 << 20) + 2)), EINVAL),
    (lambda: _norm(y_dt=1, y=P((1 << 20) + 1)), EINVAL), (lambda: _norm(eps=-1.0), EINVAL),
    (lambda: _norm(eps=float("nan")), EINVAL), (lambda: _norm(eps=float("inf")), EINVAL),
    (lambda: _norm_grad(y_dt=3), EDTYPE), (lambda: _norm_grad(s_dy=-8), EINVAL), (lambda: _norm_grad(dy=NULL), EINVAL),
    (lambda: _norm_grad(mean=NULL), EINVAL), (lambda: _norm_grad(rstd=NULL), EINVAL),
    (lambda: _norm_grad(ws=NULL), EINVAL), (lambda: _norm_grad(n=8), EINVAL),
    (lambda: _norm_grad(ws=P((1 << 21) + 8)), EINVAL), (lambda: _norm_grad(digits=P((1 << 21) + 4)), EINVAL),
    (lambda: _norm_grad(dx=P((1 << 21) + 2)), EINVAL),
    (lambda: _score(dt=2), EDTYPE), (lambda: _score(V=0), EINVAL), (lambda: _score(V=(1 << 24) + 1), EINVAL),
    (lambda: _score(N=-2), EINVAL), (lambda: _score(N=(1 << 22) + 1), EINVAL), (lambda: _score(s=-8), EINVAL),
    (lambda: _score(scale=0.0), EINVAL), (lambda: _score(scale=-1.0), EINVAL),
    (lambda: _score(scale=float("nan")), EINVAL), (lambda: _score(scale=1e6), EINVAL),
    (lambda: _score(top=-1), EINVAL), (lambda: _score(top=65, V=100), EINVAL), (lambda: _score(top=9), EINVAL),
    (lambda: _score(z=NULL), EINVAL), (lambda: _score(stat=NULL), EINVAL), (lambda: _score(lp=NULL), EINVAL),
    (lambda: _score(ti=NULL), EINVAL), (lambda: _score(tl=NULL), EINVAL), (lambda: _score(s_t=-1), EINVAL),
    (lambda: _score(stat=P((1 << 21) + 8)), EINVAL), (lambda: _score(target=P((1 << 20) + 4)), EINVAL),
    (lambda: _score(z=P((1 << 20) + 2)), EINVAL), (lambda: _score(lp=P((1 << 21) + 2)), EINVAL),
    (lambda: _score_grad(s_dz=7), EINVAL), (lambda: _score_grad(target=NULL), EINVAL),
    (lambda: _score_grad(stat=NULL), EINVAL), (lambda: _score_grad(dz=NULL), EINVAL),
    (lambda: _score_grad(s_glp=-1), EINVAL), (lambda: _score_grad(top=3, gtop=A), EINVAL),
    (lambda: _score_grad(dt=9), EDTYPE),
    (lambda: _distill(T=0.0), EINVAL), (lambda: _distill(T=-1.0), EINVAL), (lambda: _distill(T=float("nan")), EINVAL),
    (lambda: _distill(T=1e7), EINVAL), (lambda: _distill(tdt=5), EDTYPE), (lambda: _distill(K=0), EINVAL),
    (lambda: _distill(K=1025), EINVAL), (lambda: _distill(t=NULL), EINVAL), (lambda: _distill(i=NULL), EINVAL),
    (lambda: _distill(i=P((1 << 20) + 4)), EINVAL), (lambda: _distill(q=NULL), EINVAL),
    (lambda: _distill(loss=NULL), EINVAL), (lambda: _distill(s_t=-3), EINVAL),
    (lambda: _distill_grad(T=0.0), EINVAL), (lambda: _distill_grad(K=0), EINVAL), (lambda: _distill_grad(g=NULL), EINVAL),
    (lambda: _distill_grad(s_g=-1), EINVAL), (lambda: _distill_grad(s_dz=4), EINVAL),
])
def test_c_entry_points_refuse(call, want):
    assert call() == want
    assert _lib.last_error()


def test_empty_problems_are_no_ops():
    assert _norm(N=0, x=NULL, y=NULL) == _lib.DET_OK
    assert _norm_grad(N=0, dw=None, db=None, dx=NULL, ws=NULL, n=0) == _lib.DET_OK
    assert _score(N=0, z=NULL, stat=NULL) == _lib.DET_OK
    assert _score_grad(N=0) == _lib.DET_OK
    assert _distill(N=0, loss=NULL) == _lib.DET_OK


def test_workspace_sizes():
    lib = _lib.load()
    # rows that fill the chip alone, or fit one group of chunks, need none
    assert lib.det_head_workspace_bytes(4096, 131072, 0) == 0
    assert lib.det_head_workspace_bytes(1, 4 * 2048, 20) == 0
    # 64 chunks of 12 bytes, 16 workgroups of four waves' 20 keys
    assert lib.det_head_workspace_bytes(1, 131072, 20) == 64 * 12 + 64 * 20 * 8
    # alternatives: at most 16 workgroups to a row
    assert lib.det_head_workspace_bytes(1, 1 << 20, 1) == 512 * 12 + 64 * 8
    assert lib.det_head_workspace_bytes(1, 0, 0) == 0 and lib.det_head_workspace_bytes(1, 100, 65) == 0
    # chunk sums of dw and db: 64 rows to a chunk, 16 from 513 columns, 32 from 4097
    assert lib.det_layer_norm_grad_workspace_bytes(65, 512) == 2 * 2 * 512 * 4
    assert lib.det_layer_norm_grad_workspace_bytes(65, 4096) == 5 * 2 * 4096 * 4
    assert lib.det_layer_norm_grad_workspace_bytes(65, 4100) == 3 * 2 * 4100 * 4
    assert lib.det_layer_norm_grad_workspace_bytes(0, 4096) == 0


META = dict(device="meta")


def _m(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, **META)


@pytest.mark.parametrize("call,match", [
    (lambda: det.layer_norm(_m(2, 4, dtype=torch.float16)), "float32 or bfloat16"),
    (lambda: det.layer_norm(torch.empty(2, 4)), "GPU"),
    (lambda: det.layer_norm(_m(2, 0)), "at least 1"),
    (lambda: det.layer_norm(_m()), "at least 1"),
    (lambda: det.layer_norm(_m(2, 32769)), "32768"),
    (lambda: det.layer_norm(_m(2, 4), _m(5)), "weight"),
    (lambda: det.layer_norm(_m(2, 4), _m(4), _m(4, dtype=torch.bfloat16)), "share"),
    (lambda: det.layer_norm_backward(_m(2, 5), _m(2, 4), None, _m(2), _m(2)), "GPU|dy"),
    (lambda: det.DetLayerNorm(0), "features"),
    (lambda: det.DetLayerNorm(4, dtype=torch.float16), "float32"),
    (lambda: det.DetLayerNorm(4, eps=-1.0), "eps"),
    (lambda: det.token_logprobs(_m(2, 8, dtype=torch.float64)), "float32 or bfloat16"),
    (lambda: det.token_logprobs(_m(2, 8), scale=0.0), "scale"),
    (lambda: det.token_logprobs(_m(2, 8), top=9), "top"),
    (lambda: det.token_logprobs(_m(2, 100), top=65), "top"),
    (lambda: det.token_logprobs(_m(2, 8), _m(2, dtype=torch.int32)), "int64"),
    (lambda: det.token_logprobs(_m(2, 8), _m(3, dtype=torch.int64)), "shape"),
    (lambda: det.token_logprobs(torch.empty(2, 8), torch.zeros(2, dtype=torch.int64)), "GPU"),
    (lambda: det.token_logprobs(_m(2, 0)), "V"),
    (lambda: det.token_logprobs_backward(_m(2, 8), None, _m(2, 4), g_logprob=_m(2)), "targets"),
    (lambda: det.token_logprobs_backward(_m(2, 8), None, _m(3, 4)), "stat"),
    (lambda: det.distill_loss(_m(2, 8), _m(2, 3), _m(2, 3, dtype=torch.int64), temperature=0.0), "temperature"),
    (lambda: det.distill_loss(_m(2, 8), _m(3, 3), _m(3, 3, dtype=torch.int64)), "teacher"),
    (lambda: det.distill_loss(_m(2, 8), _m(2, 3), _m(2, 4, dtype=torch.int64)), "indices"),
    (lambda: det.distill_loss(_m(2, 8), _m(2, 3), _m(2, 3)), "int64"),
    (lambda: det.distill_loss(_m(2, 2000), _m(2, 1025), _m(2, 1025, dtype=torch.int64)), "1024"),
    (lambda: det.exact_mean(_m(3, dtype=torch.float16)), "float32 or bfloat16"),
])
def test_python_layer_refuses(call, match):
    with pytest.raises(ValueError, match=match):
        call()


def test_non_tensors_are_type_errors():
    with pytest.raises(TypeError):
        det.layer_norm([1.0])
    with pytest.raises(TypeError):
        det.token_logprobs([1.0])


def test_layer_norm_module():
    m = det.DetLayerNorm(6, bias=False)
    assert m.bias is None and m.weight.tolist() == [1.0] * 6 and "bias=False" in repr(m)
    m = det.DetLayerNorm(6, dtype=torch.bfloat16)
    assert m.bias.dtype == torch.bfloat16 and m.bias.tolist() == [0.0] * 6
