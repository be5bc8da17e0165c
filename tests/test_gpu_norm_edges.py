"""Layer norm's gradients where their rounding shows: bf16 sums over rows at
ties, and rows whose offset is large beside their spread."""
from fractions import Fraction

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.test_gpu_norm import _check_backward, _formula, _inputs

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


def _far_inputs(N, C, xt, yt, offset, seed):
    """Rows by turns around 0, around the offset and around its negative."""
    x, w, b, dy = _inputs(N, C, F32, yt, yt, seed)
    sign = torch.tensor([0.0, 1.0, -1.0], device="cuda")[torch.arange(N, device="cuda") % 3]
    return (x + offset * sign[:, None]).to(xt), w, b, dy


def _check_far(x, w, dy, grads, wt):
    # Derived before the first run: the mean's rounding moves h by u |mean| rstd,
    # at most 16 u in rows that keep it; the others give up the mean of h, a sum
    # like those of test_gpu_norm.py, whose bounds hold with 16 u in the place of
    # u |mean| rstd.
    q = _formula(x, w, None, dy, 1e-5)
    q["mean"] = 16.0 / q["r"]
    _check_backward(*grads, q, x.dtype, wt)


@pytest.mark.parametrize("C", [17, 130, 256, 300, 512, 1000, 1024, 1537, 4096, 5000, 8192, 12995, 16384, 20000])
@pytest.mark.parametrize("xt,yt,offset", [(F32, F32, 1.0e3), (F32, F32, 3.0e4), (F32, BF16, 3.0e6), (BF16, BF16, 300.0)],
                         ids=["f32 1e3", "f32 3e4", "f32-bf16 3e6", "bf16 300"])
def test_gradients_of_rows_far_from_zero_keep_their_precision(C, xt, yt, offset):
    N = 70
    x, w, b, dy = _far_inputs(N, C, xt, yt, offset, 300 + C)
    _, mean, rstd = det.layer_norm_forward(x, w, b, out_dtype=yt)
    grads = det.layer_norm_backward(dy, x, w, mean, rstd)
    _check_far(x, w, dy, grads, yt)
    # a row has the same bits alone; the sums the same without dx
    for rows in (slice(0, 1), slice(1, 2), slice(3, 40), slice(69, 70)):
        dx = det.layer_norm_backward(dy[rows], x[rows], w, mean[rows], rstd[rows])[0]
        assert torch.equal(dx, grads[0][rows])
    assert all(torch.equal(a, b) for a, b in zip(
        det.layer_norm_backward(dy, x, w, mean, rstd, need_dx=False)[1:], grads[1:]))
    # shards compose
    dw, db, digits = det.layer_norm_backward(dy, x, w.float(), mean, rstd, digits=True)[1:]
    parts = [det.layer_norm_digits(dy[s], x[s], mean[s], rstd[s]) for s in (slice(64, 70), slice(0, 64))]
    assert torch.equal(det.det_combine(parts), digits)
    assert torch.equal(det.det_finalize(digits), torch.stack([dw, db]))


def test_a_constant_row_far_from_zero():
    x = torch.full((5, 300), 4096.5, device="cuda")
    dy = torch.randn(5, 300, device="cuda")
    _, mean, rstd = det.layer_norm_forward(x)
    dx, dw, db = det.layer_norm_backward(dy, x, None, mean, rstd)
    assert torch.equal(dw, torch.zeros(300, device="cuda"))
    want = rstd.double()[:, None] * (dy.double() - dy.double().mean(1, keepdim=True))
    u = 2.0 ** -24
    assert ((dx.double() - want).abs() <= rstd.double()[:, None] * (64 * u * dy.double().abs().mean(1, keepdim=True)
                                                                   + 4 * u * dy.double().abs()) + 2 * u * want.abs()).all()
