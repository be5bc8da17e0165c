"""Rows of the scores and of distillation at the edges of what is defined:
teachers that are not finite, invalid entries, rows without a token under
incoming gradients that are not finite, rows that several workgroups share.

Tolerances are those of test_gpu_head.py, whose derivation they use.
"""
import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce
from tests.test_gpu_head import _check_grad, _close, _logits, _teacher, _want_distill

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
