"""Layer norm's gradients where their rounding shows: bf16 sums over rows at
ties, and rows whose offset is large beside their spread."""
from fractions import Fraction

import pytest
import torch

import bitwise_deterministic_exact_amd as det

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _bf16(v: Fraction) -> float:
    """v rounded once to bf16 (nearest, ties to even), as a float."""
    m = abs(v)
    if m == 0:
        return 0.0
    e = m.numerator.bit_length() - m.denominator.bit_length()
    e -= m < Fraction(2) ** e                                   # 2^e <= m < 2^(e + 1)
    step = Fraction(2) ** max(e - 7, -133)
    r = round(m / step) * step                                  # Fraction: ties to even
    r = float("inf") if r >= Fraction(2) ** 128 else float(r)
    return -r if v < 0 else r


def test_bf16_sums_over_rows_are_rounded_once():
    # two chunks each (rows 0 and 99).  By way of fp32: 1 + 2^-8 + 2^-30 becomes
    # 1 + 2^-8, a tie, and that 1; the nearest bf16 is 1 + 2^-7
    u = 2.0 ** -8
    cases = [(1.0, u), (1.0 + 2 * u, u), (1.0 + u, 2.0 ** -30), (1.0 + 2 * u + u, -(2.0 ** -40)), (1.0 + u, -(2.0 ** -60)),
             (-1.0 - u, -(2.0 ** -30)), (1.0 - u / 2, 2.0 ** -50), (255.5, 2.0 ** -100), (255.0, 0.0), (3.39e38, 2.0e35),
             (3.3895e38, 1.0e36), (-3.4e38, -3.0e38), (5.5, -5.5), (2.0 ** -133, 2.0 ** -134),
             (2.0 ** -133, 2.0 ** -134 + 2.0 ** -149), (2.0 ** -134, 0.0), (2.0 ** -134, 2.0 ** -149), (2.0 ** -149, 0.0),
             (-(2.0 ** -149), 0.0), (2.0 ** -126, -(2.0 ** -134)), (2.0 ** -126, -(2.0 ** -149)), (2.0 ** 100, 2.0 ** -100),
             (2.0 ** 100 * (1 + u), 2.0 ** -149), (2.0 ** 100 * (1 + u), -(2.0 ** -149)), (0.0, -0.0)]
    g = torch.Generator().manual_seed(51)
    near = (1 + torch.randint(0, 128, (200,), generator=g) / 128.0 + 2.0 ** -8) * 2.0 ** torch.randint(-140, 120, (200,), generator=g)
    cases += [(a, a * 2.0 ** -31 * s) for a in near.tolist() for s in (1.0, -1.0)]
    C = len(cases)
    dy = torch.zeros(100, C, device="cuda")
    dy[0] = torch.tensor([a for a, _ in cases])
    dy[99] = torch.tensor([b for _, b in cases])
    x = torch.randn(100, C, device="cuda")
    _, mean, rstd = det.layer_norm_forward(x)
    db = det.layer_norm_backward(dy, x, None, mean, rstd, grad_dtype=BF16)[2]
    rows = dy[[0, 99]].cpu().tolist()
    want = torch.tensor([_bf16(Fraction(a) + Fraction(b)) for a, b in zip(*rows)])
    assert torch.equal(want.to(BF16).float(), want)             # the oracle's values are bf16
    assert db.dtype == BF16 and torch.equal(db.float().cpu(), want)


def test_bf16_sums_of_many_rows_are_rounded_once():
    # enough chunks that several workgroups share a column
    C = 24
    dy = torch.zeros(140000, C, device="cuda")
    dy[5], dy[70000], dy[139999] = 1.0, 2.0 ** -8, 2.0 ** -30
    dy[:, C // 2:] *= -1
    x = torch.randn(140000, C, device="cuda")
    _, mean, rstd = det.layer_norm_forward(x)
    db = det.layer_norm_backward(dy, x, None, mean, rstd, grad_dtype=BF16)[2].float()
    assert torch.equal(db.abs(), torch.full((C,), 1.0 + 2.0 ** -7, device="cuda")) and (db[C // 2:] < 0).all()
