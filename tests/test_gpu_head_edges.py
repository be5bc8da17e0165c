"""Rows of the scores and of distillation at the edges of what is defined:
teachers that are not finite, invalid entries, rows without a token under
incoming gradients that are not finite, rows that several workgroups share.

Tolerances are those of test_gpu_head.py, whose derivation they use.
"""
import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce
from tests.test_gpu_head import _check_grad, _logits, _teacher, _want_distill

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NAMES = {F32: "f32", BF16: "bf16"}
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("N,V,K", [(6, 5, 2), (6, 5000, 8), (6, 9001, 100)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
def test_a_bad_teacher_row_has_no_finite_gradient(N, V, K, dt):
    z, _ = _logits(N, V, dt, 41)
    teacher, idx = _teacher(N, V, K, 42)
    g = torch.ones(N, device="cuda")
    clean = det.distill_backward(z, idx, *det.distill_forward(z, teacher, idx)[1:], g)
    teacher[1, 0], teacher[3, K - 1] = NAN, INF
    teacher[4, 1] = NAN
    idx[4] = -1                                    # and nothing but invalid entries
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[[1, 3, 4]] = True
    det.device_status()
    loss, stat, q = det.distill_forward(z, teacher, idx)
    dz = det.distill_backward(z, idx, stat, q, g)
    assert torch.isnan(loss[bad]).all() and torch.isnan(dz[bad]).all()
    assert torch.isfinite(loss[~bad]).all() and torch.equal(dz[~bad], clean[~bad])
    assert det.device_status() == {"nonfinite"}


@pytest.mark.parametrize("N,V,K", [(8, 5, 2), (8, 5000, 8), (8, 9001, 100), (8, 20000, 9)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
def test_an_invalid_entry_leaves_its_row_without_a_gradient(N, V, K, dt):
    z, _ = _logits(N, V, dt, 43)
    teacher, idx = _teacher(N, V, K, 44)
    g = torch.ones(N, device="cuda")
    clean = det.distill_backward(z, idx, *det.distill_forward(z, teacher, idx)[1:], g)
    idx[1, 0], idx[2, K - 1], idx[4] = V, -1, V + 3          # one, one, all of them
    teacher[6, 0], idx[6, 0] = -INF, -5                      # not there: not looked at
    teacher[7, 1], idx[7, 1] = teacher[7, 0] - 102.0, -5     # e^-102: subnormal in fp32, but there
    lost = torch.zeros(N, dtype=torch.bool, device="cuda")
    lost[[1, 2, 4, 7]] = True
    det.device_status()
    loss, stat, q = det.distill_forward(z, teacher, idx)
    dz = det.distill_backward(z, idx, stat, q, g)
    assert torch.isnan(loss[lost]).all() and torch.isfinite(loss[~lost]).all()
    assert torch.equal(q[lost], torch.zeros_like(q[lost]))
    assert torch.equal(dz[lost], torch.zeros_like(dz[lost]))
    same = ~lost
    same[6] = False
    assert torch.equal(dz[same], clean[same])
    _, _, want, tol = _want_distill(z[6:7], teacher[6:7], idx[6:7], 1.0, g[6:7])
    _check_grad(dz[6:7], want, tol, dt)
    assert det.device_status() == set()
    zr = z.clone().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(det.distill_loss(zr, teacher, idx), zr, g)[0], dz)


@pytest.mark.parametrize("V", [5, 3000, 20000])
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
@pytest.mark.parametrize("g", [INF, -INF, NAN])
def test_rows_without_a_token_have_no_gradient_whatever_comes_in(V, dt, g):
    N = 5
    z, t = _logits(N, V, dt, 45)
    z[1], z[3] = -INF, -INF
    r, stat = det.token_logprobs_forward(z, t, top=2)
    one = torch.ones(N, device="cuda")
    come = one.clone()
    come[[1, 3]] = g
    two = come[:, None].expand(N, 2)
    for kw in ({"g_logprob": come}, {"g_entropy": come}, {"g_top": two},
               {"g_logprob": come, "g_entropy": come, "g_top": two}):
        dz = det.token_logprobs_backward(z, t, stat, top_index=r.top_index, **kw)
        want = det.token_logprobs_backward(z, t, stat, top_index=r.top_index,
                                           **{k: torch.ones_like(v) for k, v in kw.items()})
        assert torch.isfinite(want).all() and torch.equal(dz, want)
        assert torch.equal(dz[[1, 3]], torch.zeros_like(dz[:2]))
    teacher, idx = _teacher(N, V, 3, 46)
    _, stat, q = det.distill_forward(z, teacher, idx)
    dz = det.distill_backward(z, idx, stat, q, come)
    assert torch.equal(dz, det.distill_backward(z, idx, stat, q, one))
    assert torch.equal(dz[[1, 3]], torch.zeros_like(dz[:2]))


# ------------------------------------------------------------ distillation's gradient, entry by entry

def _check_distill_grad(dz, z, teacher, idx, T, g):
    """_want_distill's bound; the K values that may be added at one token count
    where they are added, at the entries (off them the bound is p's alone)."""
    _, _, want, tol = _want_distill(z, teacher, idx, T, g)
    q = torch.softmax(teacher.double() / T, -1)
    own = torch.zeros_like(want).scatter_add_(-1, torch.where(q > 0, idx, 0), q)
    _check_grad(dz, want, tol + idx.shape[-1] * 2.0 ** -24 * T * g.abs().double()[:, None] * own, z.dtype)
    off = own == 0
    assert (tol[off] <= want[off].abs() / 64 + 2.0 ** -125).all()   # so a 0 in the place of p_j does not pass


@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 5, 4), (2, 2049, 7), (1, 50257, 64), (5, 8193, 33), (1030, 700, 20),
                                   (1100, 9000, 64), (3, 4000, 1000), (2, 5, 40)])
@pytest.mark.parametrize("dt,tdt", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=lambda t: NAMES[t])
@pytest.mark.parametrize("T", [1.0, 2.5])
def test_distillation_gradient_of_every_token(N, V, K, dt, tdt, T):
    announce(f"distill gradient {N}x{V} K={K} {NAMES[dt]} teacher {NAMES[tdt]} T={T}")
    z, _ = _logits(N, V, dt, N + V)
    teacher, idx = _teacher(N, V, K, K, tdt)
    g = torch.rand(N, device="cuda") - 0.3
    _, stat, q = det.distill_forward(z, teacher, idx, temperature=T)
    _check_distill_grad(det.distill_backward(z, idx, stat, q, g, temperature=T), z, teacher, idx, T, g)
