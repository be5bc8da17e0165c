"""Token log probabilities and distillation on the GPU against the formulas in
64 bits: vocabularies on both sides of every chunk and vector boundary, odd
rows, masks, ties, ignored and invalid tokens, repeated entries, strides.

Tolerances, derived before the first run.  u = 2^-24.  An exponential's
argument d = scale (z - max) carries three roundings (difference, scale,
product), so e^d is within (3 |d| + 3) u of its value, weighted by e^d itself:
at most 3 u sum p|d| + 3 u of the whole sum, p|d| summing to at most ln V + 1.
Adding 32 values per lane and 6 levels of lanes is within 38 u; the rest is in
64 bits.  So ln S is within (3 (ln V + 1) + 41) u < 96 u for V <= 2^24, a log
probability within 96 u + u |l|; the entropy, whose second sum carries the
same factors times |d|, within 96 u (2 + H) + u H.  A probability adds its own
exponent's 3 |d| u, the stored 1/S and two products: (3 |d| + 8 + 96) u of its
value, and the gradient's entropy factor (H + l) is within 8 u (2 + |l| + H).
"""
import math

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
NAMES = {F32: "f32", BF16: "bf16"}
INF = float("inf")
# (rows, vocabulary): one token, vectors and chunks (2048) and groups of four
# chunks (8192) cut at every offset, one row over several workgroups, many rows
SIZES = [(1, 1), (3, 2), (5, 7), (9, 8), (2, 255), (4, 2047), (3, 2048), (5, 2049), (2, 4097), (1, 6145), (3, 8192),
         (2, 8193), (1, 50257), (7, 32768), (1, 131072), (1030, 1001), (1100, 8195)]


def half_step(t):
    return torch.finfo(t).eps / 2


def _logits(N, V, dt, seed, masked=False):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, V, generator=g) * 3
    z[torch.arange(N), torch.randint(0, V, (N,), generator=g)] += 5
    if masked and V > 1:
        z[:, torch.rand(V, generator=g) < 0.2] = -INF
        z[:, 0] = 0.25
    t = torch.randint(0, V, (N,), generator=g)
    return z.to(dt).cuda(), t.cuda()


def _exact(z, scale):
    """(l, p, H, d, masked) of the rows in 64 bits; empty rows as documented."""
    Z = z.double()
    masked = torch.isneginf(Z)
    empty = masked.all(-1, keepdim=True)
    m = torch.where(empty, 0.0, Z.amax(-1, keepdim=True))
    d = (Z - m) * scale
    S = torch.where(empty, 1.0, d.exp().sum(-1, keepdim=True))
    l = d - S.log()
    p = l.exp()
    H = -(p * torch.where(masked, 0.0, l)).sum(-1)
    return l, p, H, d, masked


def _close(name, got, want, tol):
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin].double(), want[~fin]), f"{name}: non-finite values differ"
    err, tol = (got.double() - want).abs()[fin], (tol.expand_as(want) if torch.is_tensor(tol) else
                                                  torch.full_like(want, tol))[fin]
    assert torch.isfinite(got[fin]).all(), name
    assert not (err > tol).any(), f"{name}: worst ratio {(err / tol).max().item():.3g}"


def _top(z, k):
    # stable: ties stay in index order; -0 and +0 compare equal
    return torch.sort(z.double(), dim=-1, descending=True, stable=True).indices[..., :k]


def _check_scores(r, z, t, scale, top):
    l, p, H, d, masked = _exact(z, scale)
    lt = l.gather(-1, t[..., None])[..., 0]
    _close("logprob", r.logprob, lt, 96 * U + U * torch.nan_to_num(lt.abs(), posinf=0.0))
    _close("entropy", r.entropy, H, 96 * U * (2 + H) + U * H)
    assert (r.entropy >= 0).all()
    if top:
        i = _top(z, top)
        assert torch.equal(r.top_index, i)
        li = l.gather(-1, i)
        _close("top_logprob", r.top_logprob, li, 96 * U + U * torch.nan_to_num(li.abs(), posinf=0.0))


def _want_grad(z, t, scale, glp, gent, ti=None, gtop=None, ignore=-100):
    l, p, H, d, masked = _exact(z, scale)
    own = torch.zeros_like(l)
    if glp is not None:
        ok = t != ignore
        own.scatter_add_(-1, torch.where(ok, t, 0)[..., None], torch.where(ok, glp, 0.0).double()[..., None])
    if gtop is not None:
        own.scatter_add_(-1, ti, gtop.double())
    G = own.sum(-1, keepdim=True)
    ge = gent.double()[..., None] if gent is not None else 0.0
    l0 = torch.where(masked, 0.0, l)
    want = scale * (own - p * (G + ge * (H[..., None] + l0)))
    mass = own.abs().sum(-1, keepdim=True) + abs(ge) * (H[..., None] + l0.abs() + 2)
    d0 = torch.nan_to_num(d.abs(), posinf=0.0)
    tol = scale * (p * mass * (3 * d0 + 112) * U + 4 * U * own.abs()) + 2.0 ** -126
    empty = masked.all(-1, keepdim=True)
    return torch.where(empty, 0.0, want), tol


def _check_grad(dz, want, tol, dt):
    _close("dz", dz, want, tol + half_step(dt) * (want.abs() + tol))


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
@pytest.mark.parametrize("masked,scale", [(False, 1.0), (True, 0.7)])
def test_scores_and_gradients(N, V, dt, masked, scale):
    top = min(V, (0, 1, 5, 20, 64)[(N + V) % 5])
    announce(f"token_logprobs {N}x{V} {NAMES[dt]} top={top} masked={masked}")
    z, t = _logits(N, V, dt, 7 * N + V, masked)
    r, stat = det.token_logprobs_forward(z, t, scale=scale, top=top)
    _check_scores(r, z, t, scale, top)
    g = torch.Generator().manual_seed(3)
    glp, gent = torch.randn(N, generator=g).cuda(), (0.1 * torch.randn(N, generator=g)).cuda()
    gtop = torch.randn(N, top, generator=g).cuda() if top else None
    for a, b, c in ((glp, None, None), (None, gent, None), (glp, gent, gtop)):
        dz = det.token_logprobs_backward(z, t, stat, scale=scale, top_index=r.top_index, g_logprob=a, g_entropy=b,
                                         g_top=c)
        assert dz.dtype == dt
        _check_grad(dz, *_want_grad(z, t, scale, a, b, r.top_index, c), dt)
    # autograd gives the same bits
    zr = z.clone().requires_grad_(True)
    ra = det.token_logprobs(zr, t, scale=scale, top=top)
    assert torch.equal(ra.logprob, r.logprob) and torch.equal(ra.top_index, r.top_index)
    outs, grads = [ra.logprob, ra.entropy], [glp, gent]
    if top:
        outs.append(ra.top_logprob)
        grads.append(gtop)
    got, = torch.autograd.grad(outs, zr, grads)
    assert torch.equal(got, dz)


@pytest.mark.parametrize("N,V", [(1, 131072), (3, 8193), (1100, 8195), (1030, 900)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
@pytest.mark.parametrize("kind", ["constant", "ascending", "descending", "period", "signed zeros", "lowest"])
def test_alternatives_of_adversarial_rows(N, V, dt, kind):
    # ties everywhere, every chunk better than the one before, the best
    # elements all in a few lanes, -0 among +0, masks of the lowest finite value
    i = torch.arange(V)
    row = {"constant": torch.full((V,), 1.5), "ascending": (i // 97).float() * 0.01,
           "descending": -(i // 97).float() * 0.01, "period": torch.where(i % 512 < 8, 4.0 + (i // 512) * 0.001, 0.0),
           "signed zeros": torch.where(i % 3 == 0, -0.0, 0.0),
           "lowest": torch.where(i % 5 == 1, (i % 7).float(), torch.finfo(dt).min)}[kind]
    z = row.to(dt).expand(N, V).contiguous().cuda()
    t = torch.arange(N, device="cuda") % V
    for top in (1, 20, 64):
        announce(f"alternatives {kind} {N}x{V} {NAMES[dt]} top={top}")
        r = det.token_logprobs(z, t, top=top)
        assert torch.equal(r.top_index, _top(z[:1], top).expand(N, top))
    if kind != "lowest":
        _check_scores(r, z, t, 1.0, 64)
    else:
        l, p, H, d, _ = _exact(z, 1.0)
        _close("entropy", r.entropy, H, 96 * U * (2 + H))
        _close("logprob", r.logprob, l.gather(-1, t[:, None])[:, 0], 96 * U + 2 * U * l.abs().gather(-1, t[:, None])[:, 0])


def test_rows_of_the_lowest_value_are_uniform():
    for dt in (F32, BF16):
        z = torch.full((2, 5000), torch.finfo(dt).min, dtype=dt, device="cuda")
        r = det.token_logprobs(z, torch.tensor([3, 4999], device="cuda"), top=3)
        want = torch.full((2,), -math.log(5000), dtype=torch.float64, device="cuda")
        _close("logprob", r.logprob, want, 96 * U + U * 10)
        _close("entropy", r.entropy, -want, 96 * U * 12)
        assert r.top_index.tolist() == [[0, 1, 2]] * 2


@pytest.mark.parametrize("N,V", [(4, 37), (3, 20000), (1030, 2500)])
@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
def test_empty_and_nearly_empty_rows(N, V, dt):
    z, t = _logits(N, V, dt, 11)
    z[1] = -INF                                   # nothing left
    z[2] = -INF
    z[2, V - 1] = -3.0                            # one token left
    t[2] = V - 1
    det.device_status()
    r, stat = det.token_logprobs_forward(z, t, top=5)
    _check_scores(r, z, t, 1.0, 5)
    assert r.logprob[1] == -INF and r.entropy[1] == 0 and (r.top_logprob[1] == -INF).all()
    assert r.top_index[1].tolist() == [0, 1, 2, 3, 4]
    assert r.logprob[2] == 0 and r.entropy[2] == 0 and r.top_index[2].tolist() == [V - 1, 0, 1, 2, 3]
    one = torch.ones(N, device="cuda")
    dz = det.token_logprobs_backward(z, t, stat, g_logprob=one, g_entropy=one)
    assert torch.equal(dz[1], torch.zeros_like(dz[1])) and torch.isfinite(dz).all()
    _check_grad(dz, *_want_grad(z, t, 1.0, one, one), dt)
    assert det.device_status() == set()


@pytest.mark.parametrize("N,V", [(6, 50), (6, 30000), (1040, 3000)])
def test_nan_and_inf_rows(N, V):
    z, t = _logits(N, V, F32, 12)
    clean = det.token_logprobs(z, t, top=7)
    det.device_status()
    z[0, V // 2], z[3, V - 1], z[4] = float("nan"), INF, float("nan")
    r, stat = det.token_logprobs_forward(z, t, top=7)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[[0, 3, 4]] = True
    for got, was in ((r.logprob, clean.logprob), (r.entropy, clean.entropy), (r.top_logprob, clean.top_logprob)):
        assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], was[~bad])
    assert (r.top_index[bad] == -1).all() and torch.equal(r.top_index[~bad], clean.top_index[~bad])
    dz = det.token_logprobs_backward(z, t, stat, g_logprob=torch.ones(N, device="cuda"), top_index=r.top_index,
                                     g_top=torch.ones(N, 7, device="cuda"))
    assert torch.isnan(dz[bad]).all() and torch.isfinite(dz[~bad]).all()
    assert det.device_status() == {"nonfinite"}


def test_ignored_and_invalid_targets():
    z, t = _logits(5, 3000, F32, 13)
    t[1], t[2], t[3] = -100, -7, 3000
    zr = z.clone().requires_grad_(True)
    r = det.token_logprobs(zr, t)
    assert r.logprob[1] == 0 and torch.isnan(r.logprob[2:4]).all() and torch.isfinite(r.logprob[[0, 4]]).all()
    dz, = torch.autograd.grad(r.logprob, zr, torch.ones(5, device="cuda"))
    assert torch.equal(dz[1:4], torch.zeros_like(dz[1:4])) and dz[0].abs().sum() > 0
    # an ignored token inside the vocabulary
    t = torch.zeros(5, dtype=torch.int64, device="cuda")
    r, stat = det.token_logprobs_forward(z, t, ignore_index=0)
    assert torch.equal(r.logprob, torch.zeros(5, device="cuda"))
    dz = det.token_logprobs_backward(z, t, stat, ignore_index=0, g_logprob=torch.ones(5, device="cuda"))
    assert torch.equal(dz, torch.zeros_like(dz))
    # no targets at all
    r = det.token_logprobs(z, top=2)
    assert r.logprob is None and torch.equal(r.top_index, _top(z, 2))
    zr = z.clone().requires_grad_(True)
    r = det.token_logprobs(zr, None, top=2)
    got, = torch.autograd.grad(r.top_logprob.sum(), zr)
    _check_grad(got, *_want_grad(z, None, 1.0, None, None, r.top_index, torch.ones(5, 2, device="cuda")), F32)


@pytest.mark.parametrize("dt", [F32, BF16], ids=NAMES.get)
@pytest.mark.parametrize("V", [1000, 5001, 30000, 40000])
def test_rows_do_not_depend_on_the_batch_or_the_layout(dt, V):
    N = 1100                                       # finished in one launch; few rows share workgroups
    z, t = _logits(N, V, dt, 14)
    full, fstat = det.token_logprobs_forward(z, t, top=9)
    g = torch.randn(N, device="cuda")
    fdz = det.token_logprobs_backward(z, t, fstat, g_logprob=g, g_entropy=g)
    for rows in (slice(0, 1), slice(3, 5), slice(1099, 1100), slice(20, 220), slice(10, 310)):
        r, stat = det.token_logprobs_forward(z[rows], t[rows], top=9)
        for a, b in zip(r, full):
            assert torch.equal(a, b[rows])
        assert torch.equal(stat, fstat[rows])
        assert torch.equal(det.token_logprobs_backward(z[rows], t[rows], stat, g_logprob=g[rows], g_entropy=g[rows]),
                           fdz[rows])
    # rows apart and misaligned; a transposed view; leading shape; strided targets
    wide = torch.zeros(N, V + 13, dtype=dt, device="cuda")
    wide[:, 5:5 + V] = z
    tt = torch.stack([t, t], dim=1)
    for zz, ts in ((wide[:, 5:5 + V], t), (z[:64].t().contiguous().t(), t[:64]), (z, tt[:, 1])):
        n = zz.shape[0]
        r, stat = det.token_logprobs_forward(zz, ts, top=9)
        for a, b in zip(r, full):
            assert torch.equal(a, b[:n])
        assert torch.equal(det.token_logprobs_backward(zz, ts, stat, g_logprob=g[:n], g_entropy=g[:n]), fdz[:n])
    r = det.token_logprobs(z.reshape(11, 100, V), t.reshape(11, 100), top=9)
    assert torch.equal(r.logprob, full.logprob.reshape(11, 100))
    assert torch.equal(r.top_index, full.top_index.reshape(11, 100, 9))
    r1 = det.token_logprobs(z[0], t[0], top=9)
    assert r1.logprob.shape == () and torch.equal(r1.logprob, full.logprob[0]) and r1.top_index.shape == (9,)


def test_broadcast_and_strided_gradients():
    z, t = _logits(6, 4100, F32, 15)
    zr = z.clone().requires_grad_(True)
    r = det.token_logprobs(zr, t, top=3)
    got, = torch.autograd.grad(r.logprob.sum() + 2 * r.entropy.sum() + r.top_logprob.sum(), zr)
    _, stat = det.token_logprobs_forward(z, t)
    one = torch.ones(6, device="cuda")
    want = det.token_logprobs_backward(z, t, stat, g_logprob=one, g_entropy=2 * one, top_index=r.top_index,
                                       g_top=torch.ones(6, 3, device="cuda"))
    assert torch.equal(got, want)
    g2 = torch.randn(6, 2, device="cuda")
    gt = torch.randn(3, 6, device="cuda").t()
    a = det.token_logprobs_backward(z, t, stat, g_logprob=g2[:, 1], top_index=r.top_index, g_top=gt)
    b = det.token_logprobs_backward(z, t, stat, g_logprob=g2[:, 1].contiguous(), top_index=r.top_index,
                                    g_top=gt.contiguous())
    assert torch.equal(a, b)


def test_far_rows_pass_32_bit_offsets():
    # rows more than 2^32 bytes apart
    V, far = 3001, (1 << 30) + 77
    base = torch.zeros(2 * far + V, dtype=BF16, device="cuda")
    z = base.as_strided((3, V), (far, 1))
    rows, t = _logits(3, V, BF16, 16)
    z.copy_(rows)
    a, sa = det.token_logprobs_forward(z, t, top=4)
    b, sb = det.token_logprobs_forward(rows, t, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and torch.equal(sa, sb)
    one = torch.ones(3, device="cuda")
    assert torch.equal(det.token_logprobs_backward(z, t, sa, g_logprob=one),
                       det.token_logprobs_backward(rows, t, sb, g_logprob=one))


def test_no_rows():
    z = torch.empty(0, 100, device="cuda", requires_grad=True)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    r = det.token_logprobs(z, t, top=3)
    assert r.logprob.shape == (0,) and r.top_index.shape == (0, 3)
    dz, = torch.autograd.grad(r.logprob.sum(), z)
    assert dz.shape == (0, 100)
    loss = det.distill_loss(z, torch.empty(0, 4, device="cuda"), torch.empty(0, 4, dtype=torch.int64, device="cuda"))
    assert loss.shape == (0,)


# ------------------------------------------------------------ distillation

def _teacher(N, V, K, seed, dt=F32):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else torch.randint(0, V, (K,), generator=g)
                       for _ in range(N)])
    return (2.5 * torch.randn(N, K, generator=g)).to(dt).cuda(), idx.cuda()


def _want_distill(z, teacher, idx, T, g):
    l, p, H, d, masked = _exact(z, 1.0 / T)
    tt = teacher.double() / T
    none = torch.isneginf(tt).all(-1, keepdim=True)
    lq = torch.where(none, -INF, torch.log_softmax(torch.where(none, 0.0, tt), -1))
    q = lq.exp()
    li = l.gather(-1, torch.where(q > 0, idx, 0))
    term = torch.where(q > 0, q * (torch.where(q > 0, lq, 0.0) - li), 0.0)
    loss = T * T * term.sum(-1)
    ltol = T * T * (96 * U + 1e-13 * term.abs().sum(-1)) + U * torch.nan_to_num(loss.abs(), posinf=0.0)
    own = torch.zeros_like(l).scatter_add_(-1, torch.where(q > 0, idx, 0), q)
    some = torch.where(none | masked.all(-1, keepdim=True), 0.0, 1.0)
    gT = g.double()[..., None] * T
    want = gT * (p * some - own * some)
    d0 = torch.nan_to_num(d.abs(), posinf=0.0)
    tol = gT.abs() * (p * (3 * d0 + 112) * U + 6 * U * own) + 2.0 ** -126
    return loss, ltol, want, tol


@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 5, 4), (2, 2049, 7), (1, 50257, 64), (5, 8193, 33), (1030, 700, 20),
                                   (1100, 9000, 64), (3, 4000, 1000), (2, 5, 40)])
@pytest.mark.parametrize("dt,tdt", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=lambda t: NAMES[t])
@pytest.mark.parametrize("T", [1.0, 2.5])
def test_distillation(N, V, K, dt, tdt, T):
    announce(f"distill {N}x{V} K={K} {NAMES[dt]} teacher {NAMES[tdt]} T={T}")
    z, _ = _logits(N, V, dt, N + V)
    teacher, idx = _teacher(N, V, K, K, tdt)       # K > V: repeated entries
    g = torch.rand(N, device="cuda") - 0.3
    loss, ltol, want, tol = _want_distill(z, teacher, idx, T, g)
    zr = z.clone().requires_grad_(True)
    got = det.distill_loss(zr, teacher, idx, temperature=T)
    _close("loss", got.detach(), loss, ltol)
    dz, = torch.autograd.grad(got, zr, g)
    # equal entries are added in fp32: K u of their sum
    _check_grad(dz, want, tol + K * U * tol.new_tensor(T) * g.abs().double()[:, None], dt)


def test_distillation_masks():
    N, V, K = 6, 5000, 8
    z, _ = _logits(N, V, F32, 17)
    teacher, idx = _teacher(N, V, K, 18)
    teacher[0] = -INF                              # no entries: loss 0, no gradient
    teacher[1, 3:] = -INF
    idx[1, 3:] = -1                                # padding that is not looked at
    z[2] = -INF                                    # a student row with nothing left
    z[3, idx[3, 2]] = -INF                         # a taught token that the student masks
    idx[4, 5] = V                                  # an invalid entry
    g = torch.ones(N, device="cuda")
    det.device_status()
    loss, stat, q = det.distill_forward(z, teacher, idx)
    dz = det.distill_backward(z, idx, stat, q, g)
    keep = [0, 1, 2, 3, 5]
    lw, ltol, want, tol = _want_distill(z[keep], teacher[keep], idx[keep], 1.0, g[keep])
    assert loss[0] == 0 and loss[2] == INF and loss[3] == INF and torch.isnan(loss[4])
    _close("loss", loss[keep], lw, ltol)
    _check_grad(dz[keep], want, tol, F32)
    assert torch.equal(dz[0], torch.zeros(V, device="cuda")) and torch.equal(dz[2], torch.zeros(V, device="cuda"))
    assert torch.isfinite(dz).all() and det.device_status() == set()
    teacher[5, 0] = float("nan")
    assert torch.isnan(det.distill_loss(z, teacher, idx)[5]) and det.device_status() == {"nonfinite"}


@pytest.mark.parametrize("V", [900, 30000])
def test_distillation_rows_do_not_depend_on_the_batch(V):
    N, K = 1100, 16
    z, _ = _logits(N, V, BF16, 19)
    teacher, idx = _teacher(N, V, K, 20)
    g = torch.rand(N, device="cuda")
    loss, stat, q = det.distill_forward(z, teacher, idx, temperature=2.0)
    dz = det.distill_backward(z, idx, stat, q, g, temperature=2.0)
    # leading shape, entries as slices of wider ones, a broadcast gradient
    tw, iw = torch.randn(N, 40, device="cuda"), torch.zeros(N, 40, dtype=torch.int64, device="cuda")
    tw[:, 7:7 + K], iw[:, 7:7 + K] = teacher, idx
    for rows in (slice(0, 1), slice(1099, 1100), slice(20, 220)):
        l1, s1, q1 = det.distill_forward(z[rows], tw[rows, 7:7 + K], iw[rows, 7:7 + K], temperature=2.0)
        assert torch.equal(l1, loss[rows]) and torch.equal(q1, q[rows])
        assert torch.equal(det.distill_backward(z[rows], iw[rows, 7:7 + K], s1, q1, g[rows], temperature=2.0), dz[rows])
    zr = z.reshape(10, 110, V).clone().requires_grad_(True)
    l3 = det.distill_loss(zr, teacher.reshape(10, 110, K), idx.reshape(10, 110, K), temperature=2.0)
    assert torch.equal(l3.detach(), loss.reshape(10, 110))
    d1, = torch.autograd.grad(l3.sum(), zr)
    assert torch.equal(d1.reshape(N, V), det.distill_backward(z, idx, stat, q, torch.ones(N, device="cuda"),
                                                              temperature=2.0))


def test_exact_mean():
    t = torch.randn(3, 1001, device="cuda", requires_grad=True)
    m = det.exact_mean(t)
    perm = torch.randperm(3003)
    assert torch.equal(det.exact_mean(t.detach().reshape(-1)[perm.cuda()]), m.detach())
    want = t.detach().double().sum().float() / torch.tensor(3003.0, device="cuda")
    assert abs(m.item() - want.item()) <= 2 * U * abs(want.item())
    g, = torch.autograd.grad(m, t)
    assert torch.equal(g, torch.full_like(t, 1.0) / 3003.0) or (g - 1 / 3003).abs().max() < 2 * U / 3003


# ------------------------------------------------------------ gradients, graphs

def test_gradients_against_differences():
    z, t = _logits(4, 60, F32, 22)
    teacher, idx = _teacher(4, 60, 5, 23)
    g = torch.rand(4, device="cuda") + 0.5
    _, stat = det.token_logprobs_forward(z, t, scale=0.8)
    ds = det.token_logprobs_backward(z, t, stat, scale=0.8, g_logprob=g, g_entropy=g)
    loss, dstat, q = det.distill_forward(z, teacher, idx, temperature=2.0)
    dd = det.distill_backward(z, idx, dstat, q, g, temperature=2.0)

    def score(Z):
        l, p, H, _, _ = _exact(Z, 0.8)
        return ((l.gather(-1, t[:, None])[:, 0] + H) * g.double()).sum()

    def distill(Z):
        l = _exact(Z, 0.5)[0].gather(-1, idx)
        lq = torch.log_softmax(teacher.double() / 2, -1)
        return (4 * (lq.exp() * (lq - l)).sum(-1) * g.double()).sum()

    e = 2.0 ** -12
    for f, grad in ((score, ds), (distill, dd)):
        v = torch.randn(4, 60, dtype=torch.float64, device="cuda")
        slope = (f(z.double() + e * v) - f(z.double() - e * v)) / (2 * e)
        want = (grad.double() * v).sum()
        # e^2 / 6 of the third derivative (at most 32 |v|^3 per row here) and the gradient's 256 u
        tol = e * e * 32 * v.abs().pow(3).sum() + 256 * U * (grad.double() * v).abs().sum()
        assert (slope - want).abs() <= tol


@pytest.mark.parametrize("N", [3, 1030])
def test_streams_repetition_and_graph_replay(N):
    V, K = 9001, 12
    z, t = _logits(N, V, BF16, 24)
    teacher, idx = _teacher(N, V, K, 25)
    g = torch.rand(N, device="cuda")

    def step(zz):
        r, stat = det.token_logprobs_forward(zz, t, top=6)
        dz = det.token_logprobs_backward(zz, t, stat, g_logprob=g, g_entropy=g)
        loss, ds, q = det.distill_forward(zz, teacher, idx, temperature=2.0)
        return (*r, dz, loss, det.distill_backward(zz, idx, ds, q, g, temperature=2.0))

    want = step(z)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(step(z), want))
    s.synchronize()
    sz = z.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(sz)
    for k in range(4):
        nz = (z.float() * (0.5 + k) - k).to(BF16)
        sz.copy_(nz)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step(nz))), k
