"""Rows of the scores and of distillation at the edges of what is defined:
teachers that are not finite, invalid entries, rows without a token under
incoming gradients that are not finite, rows that several workgroups share.

Tolerances are those of test_gpu_head.py, whose derivation they use.
"""
import math

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from bitwise_deterministic_exact_amd import _lib
from tests.gpu_util import announce
from tests.test_gpu_head import (_check_grad, _check_scores, _close, _logits, _teacher, _want_distill,
                                 _want_grad)

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


# ------------------------------------------------------------ rows that several workgroups share

# without alternatives: one to 512 workgroups' sums of a row in the workspace, by
# few rows, by 384 and more, and by rows of more chunks than one workgroup holds
SHARED = [(1, 131072), (1, 200003), (3, 70001), (300, 50257), (400, 140000), (1, (1 << 20) + 5), (2, 1 << 24)]


@pytest.mark.parametrize("N,V", SHARED)
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
def test_scores_of_rows_that_workgroups_share(N, V, dt):
    announce(f"shared rows, scores {N}x{V} {NAMES[dt]}")
    assert _lib.load().det_head_workspace_bytes(N, V, 0) > 0
    z, t = _logits(N, V, dt, 47 + N, masked=True)
    if N > 2:
        z[1] = -INF
        z[2], t[2] = -INF, V - 1
        z[2, V - 1] = 3.0
    r, stat = det.token_logprobs_forward(z, t, scale=0.7)
    _check_scores(r, z, t, 0.7, 0)
    g = torch.Generator().manual_seed(48)
    glp, gent = torch.randn(N, generator=g).cuda(), (0.1 * torch.randn(N, generator=g)).cuda()
    dz = det.token_logprobs_backward(z, t, stat, scale=0.7, g_logprob=glp, g_entropy=gent)
    _check_grad(dz, *_want_grad(z, t, 0.7, glp, gent), dt)
    for i in {0, N // 2, N - 1}:                   # alone a row has other workgroups, and the same bits
        r1, s1 = det.token_logprobs_forward(z[i:i + 1], t[i:i + 1], scale=0.7)
        assert torch.equal(s1, stat[i:i + 1]) and torch.equal(r1.logprob, r.logprob[i:i + 1])
        d1 = det.token_logprobs_backward(z[i:i + 1], t[i:i + 1], s1, scale=0.7, g_logprob=glp[i:i + 1],
                                         g_entropy=gent[i:i + 1])
        assert torch.equal(d1, dz[i:i + 1])
    if N > 2:                                      # a NaN stays in its row
        z[0, V // 3] = NAN
        det.device_status()
        r1 = det.token_logprobs(z, t, scale=0.7)
        assert torch.isnan(r1.logprob[0]) and torch.isnan(r1.entropy[0])
        assert torch.equal(r1.logprob[1:], r.logprob[1:]) and torch.equal(r1.entropy[1:], r.entropy[1:])
        assert det.device_status() == {"nonfinite"}


@pytest.mark.parametrize("N,V", SHARED)
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
def test_distillation_of_rows_that_workgroups_share(N, V, dt):
    announce(f"shared rows, distillation {N}x{V} {NAMES[dt]}")
    assert _lib.load().det_head_workspace_bytes(N, V, 0) > 0
    K, T = 100, 2.0                                # more entries than a wave has lanes
    z, _ = _logits(N, V, dt, 49 + N)
    g = torch.Generator().manual_seed(50)
    idx = torch.randint(0, V, (N, K), generator=g).cuda()
    teacher = (2.5 * torch.randn(N, K, generator=g)).cuda()
    idx[:, 70:80] = idx[:, :10]                    # repeated
    teacher[:, 90:] = -INF                         # not there, and not looked at
    idx[:, 90:] = -7
    if N > 2:
        teacher[2], idx[1, 65] = -INF, V           # no entry at all; an invalid one
    gr = torch.rand(N, generator=g).cuda() - 0.3
    loss, stat, q = det.distill_forward(z, teacher, idx, temperature=T)
    dz = det.distill_backward(z, idx, stat, q, gr, temperature=T)
    keep = [i for i in range(N) if N <= 2 or i != 1]
    lw, ltol, _, _ = _want_distill(z[keep], teacher[keep], idx[keep], T, gr[keep])
    _close("loss", loss[keep], lw, ltol)
    some = [i for i in keep if N <= 2 or i != 2]
    _check_distill_grad(dz[some], z[some], teacher[some], idx[some], T, gr[some])
    if N > 2:
        assert torch.isnan(loss[1]) and loss[2] == 0
        assert torch.equal(dz[1:3], torch.zeros_like(dz[1:3]))
    for i in {0, N // 2, N - 1}:
        l1, s1, q1 = det.distill_forward(z[i:i + 1], teacher[i:i + 1], idx[i:i + 1], temperature=T)
        assert torch.equal(l1.nan_to_num(7.0), loss[i:i + 1].nan_to_num(7.0)) and torch.equal(q1, q[i:i + 1])
        assert torch.equal(det.distill_backward(z[i:i + 1], idx[i:i + 1], s1, q1, gr[i:i + 1], temperature=T), dz[i:i + 1])


def test_many_rows_of_more_chunks_than_a_workgroup_holds():
    # 800 rows of just over 2^20 logits (four different ones, read with their own
    # targets): two workgroups to a row, where a row alone has 129
    N, V = 800, (1 << 20) + 5
    assert _lib.load().det_head_workspace_bytes(N, V, 0) > 0
    assert _lib.load().det_head_workspace_bytes(N, V - 5, 0) == 0
    four, _ = _logits(4, V, BF16, 51, masked=True)
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(52)).cuda()
    which = torch.arange(N, device="cuda") % 4
    z = four[which]
    r, stat = det.token_logprobs_forward(z, t)
    _check_scores(type(r)(r.logprob[:4], r.entropy[:4], r.top_logprob[:4], r.top_index[:4]), z[:4], t[:4], 1.0, 0)
    g = torch.rand(N, device="cuda")
    dz = det.token_logprobs_backward(z, t, stat, g_logprob=g, g_entropy=g)
    _check_grad(dz[:4], *_want_grad(z[:4], t[:4], 1.0, g[:4], g[:4]), BF16)
    for i in range(0, N, 57):
        r1, s1 = det.token_logprobs_forward(four[i % 4:i % 4 + 1], t[i:i + 1])
        assert torch.equal(s1, stat[i:i + 1]) and torch.equal(r1.logprob, r.logprob[i:i + 1])
        assert torch.equal(det.token_logprobs_backward(z[i:i + 1], t[i:i + 1], s1, g_logprob=g[i:i + 1],
                                                       g_entropy=g[i:i + 1]), dz[i:i + 1])


# ------------------------------------------------------------ exact_mean

@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
@pytest.mark.parametrize("shape", [(1,), (), (3, 1001), (64, 64), (100003,)])
def test_exact_mean_and_its_gradient_bit_for_bit(dt, shape):
    t = (torch.randn(shape, generator=torch.Generator().manual_seed(53)) * 3).to(dt)
    n = max(t.numel(), 1)
    # fsum rounds the exact sum to 64 bits, far from a tie of fp32 here
    total = torch.tensor(math.fsum(t.double().reshape(-1).tolist()), dtype=torch.float64).float()
    x = t.cuda().requires_grad_(True)
    m = det.exact_mean(x)
    assert m.shape == () and m.dtype == F32 and torch.equal(m.detach().cpu(), total / torch.tensor(float(n)))
    g, = torch.autograd.grad(3.0 * m, x)
    assert g.shape == x.shape and g.dtype == dt
    assert torch.equal(g.cpu(), (torch.tensor(3.0) / torch.tensor(float(n))).to(dt).expand(shape))
    if t.dim() == 2:
        assert torch.equal(det.exact_mean(x.detach().t()), m.detach())
        assert torch.equal(det.exact_mean(x.detach()[:, ::2]), det.exact_mean(x.detach()[:, ::2].contiguous()))


def test_exact_mean_loses_nothing_and_takes_no_elements():
    t = torch.tensor([1e30, 1.0, 2.0, -1e30], device="cuda")
    assert det.exact_mean(t).item() == 0.75
    for dt in (F32, BF16):
        x = torch.empty(0, 4, dtype=dt, device="cuda", requires_grad=True)
        m = det.exact_mean(x)
        assert m.item() == 0.0 and torch.autograd.grad(m, x)[0].shape == (0, 4)
