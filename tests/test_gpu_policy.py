"""The policy and preference losses on the GPU against 64 bits: every reduction
and kind, ragged and empty masks, borders of the clipping, order of the rows,
layouts, long rows, streams and graph replays."""
import math

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24                                      # half a step of fp32
NAN, INF = float("nan"), float("inf")
# one token, ragged vectors, rows of one wave and of one and several workgroups, more pieces than one thread adds,
# more rows than one workgroup joins
SIZES = [(1, 1), (3, 7), (8, 300), (5, 512), (4, 513), (2, 5000), (3, 9000), (1, 40000), (700, 33), (17000, 3)]


def answers(seed, B, T, per_token=True, ref=True, masked=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    lp = -torch.abs(1.5 * r(B, T))
    mask = None
    if masked:
        mask = torch.rand(B, T, generator=g, device=DEV) < 0.7
        if B > 2:
            mask[B // 2] = False
        lp = lp.masked_fill(~mask, NAN)
    old, other = lp + 0.25 * r(B, T), lp + r(B, T)
    return lp, old, r(B, T) if per_token else r(B), mask, other if ref else None


def policy64(lp, old, adv, mask, ref, low, high, beta):
    """(loss, kl, clipped, slope, loss' bound, kl's bound, slope's bound) per token."""
    z = lambda t: (t if mask is None else t.masked_fill(~mask, 0.0)).double()
    lp, old = z(lp), z(old)
    adv = (adv if adv.shape == lp.shape else adv[..., None].expand_as(lp)).double()
    d = lp - old
    r = torch.exp(d)
    clipped = ((adv > 0) & (d > math.log1p(high))) | ((adv < 0) & (d < (math.log1p(-low) if low < 1 else -INF)))
    value = torch.where(clipped, torch.where(adv > 0, 1 + high, 1 - low), r)
    loss, slope = -value * adv, torch.where(clipped, 0.0, -r * adv)
    # e^d: 2 units of the exponential and its parts, the product: 8 half steps in all
    bl = 8 * U * (value * adv).abs()
    bs = bl.clone()
    kl, bk = torch.zeros_like(loss), torch.zeros_like(loss)
    if ref is not None:
        q = z(ref) - lp
        kl, rise = torch.expm1(q) - q, torch.expm1(q)
        # near 0 a series (q rounded once: 2 half steps of q^2, 10 of the terms), else the parts' own roundings
        bk = torch.where(q.abs() <= 1.0, 12 * U * kl, (6 + 2 * q.abs()) * U * (torch.exp(q) + 1 + q.abs()))
        loss, slope = loss + beta * kl, slope - beta * rise
        bl = bl + beta * (bk + 2 * U * kl) + 2 * U * loss.abs()
        bs = bs + beta * (bk + 4 * U * (rise.abs() + q.abs().clamp(max=1.0))) + 2 * U * slope.abs()
    out = [loss, kl, clipped.double(), slope, bl, bk, bs]
    return [t if mask is None else t.masked_fill(~mask, 0.0) for t in out]


def reduce64(t, mask, reduction):
    n = torch.full(t.shape[:1], t.shape[1], device=DEV) if mask is None else mask.sum(1)
    if reduction == "tokens":
        return t.sum() / max(1, int(n.sum()))
    return (t.sum(1) / n.clamp(min=1)).sum() / max(1, int((n > 0).sum()))


def weights64(mask, shape, reduction):
    n = torch.full(shape[:1], shape[1], device=DEV) if mask is None else mask.sum(1)
    if reduction == "tokens":
        return torch.full(shape, 1.0 / max(1, int(n.sum())), dtype=torch.float64, device=DEV)
    return (1.0 / (n.clamp(min=1).double() * max(1, int((n > 0).sum()))))[:, None].expand(shape)


def within(got, want, bound, what):
    assert got.dtype == torch.float32
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off: {got[bad][:3]} for {want[bad][:3]}"


@pytest.mark.parametrize("reduction", ["tokens", "sequences", "none"])
@pytest.mark.parametrize("per_token,ref,masked", [(True, True, True), (False, False, True), (False, True, False)])
@pytest.mark.parametrize("B,T", SIZES)
def test_policy_against_64_bits(B, T, per_token, ref, masked, reduction):
    announce(f"policy {B} {T} {per_token} {ref} {masked} {reduction}")
    beta = 0.3 if ref else 0.0
    args = answers(1, B, T, per_token, ref, masked)
    lp, old, adv, mask, other = args
    loss, kl, clipped, slope, bl, bk, bs = policy64(*args, 0.2, 0.28, beta)
    lp.requires_grad_(True)
    opts = dict(ref_logprob=other, clip_low=0.2, clip_high=0.28, kl_weight=beta, reduction=reduction)
    r = det.policy_loss(lp, old, adv, mask, **opts)
    tiny = 1e-37
    if reduction == "none":
        within(r.loss, loss, bl + tiny, "loss")
        within(r.kl, kl, bk + tiny, "kl")
        assert torch.equal(r.clipped.double(), clipped)
        g = torch.randn(B, T, device=DEV)
        w = g.double()
        grad, = torch.autograd.grad(r.loss, lp, g)
    else:
        # a row's value and the sum round once each, the divisions twice
        up = lambda t, b: reduce64(b, mask, reduction) + 4 * U * reduce64(t.abs(), mask, reduction) + tiny
        for name, got, t, b in (("loss", r.loss, loss, bl), ("kl", r.kl, kl, bk), ("clipped", r.clipped, clipped, 0 * clipped)):
            assert got.shape == ()
            within(got, reduce64(t, mask, reduction), up(t, b), name)
        g = torch.tensor(1.7, device=DEV)
        w = weights64(mask, (B, T), reduction) * g.double()
        grad, = torch.autograd.grad(r.loss, lp, g)
    within(grad, slope * w, bs * w.abs() * 1.01 + 3 * U * (slope * w).abs() + tiny, "gradient")
    if mask is not None:
        assert (grad[~mask] == 0).all()
    f, count = det.policy_loss_forward(lp.detach(), old, adv, mask, **opts)
    assert all(torch.equal(a.detach(), b) for a, b in zip(r, f))
    assert torch.equal(grad, det.policy_loss_backward(g, lp.detach(), old, adv, mask, count, **opts))
    with torch.no_grad():
        assert torch.equal(det.policy_loss(lp, old, adv, mask, **opts).loss, r.loss)


def test_borders_of_the_clipping():
    # tokens whose ratio lies within 2^-30 of a bound on either side: differences of fp32 values are exact in 64 bits
    for low, high in ((0.2, 0.28), (0.0, 0.0), (1.0, 5.0)):
        for edge in (math.log1p(high), math.log1p(-low) if low < 1 else -30.0):
            old = torch.full((64,), -3.0, device=DEV)
            lp = (old.double() + edge).float()
            for k in range(-32, 32):
                lp[k + 32] = torch.tensor(lp[k + 32].item() * (1 + k * 2.0 ** -23))
            for a in (1.5, -1.5, 0.0):
                adv = torch.full((64,), a, device=DEV)
                want = policy64(lp[None], old[None], adv[None], None, None, low, high, 0.0)
                lp_ = lp.clone().requires_grad_(True)
                r = det.policy_loss(lp_, old, adv, clip_low=low, clip_high=high, reduction="none")
                g, = torch.autograd.grad(r.loss.sum(), lp_)
                assert torch.equal(r.clipped.double(), want[2][0])
                within(r.loss, want[0][0], want[4][0], "loss")
                within(g, want[3][0], want[6][0], "gradient")


@pytest.mark.parametrize("reduction", ["tokens", "sequences"])
@pytest.mark.parametrize("B,T", [(40, 300), (3000, 17), (20000, 2), (6, 9000)])
def test_the_order_of_the_rows_does_not_matter(B, T, reduction):
    lp, old, adv, mask, ref = answers(2, B, T)
    opts = dict(kl_weight=0.1, reduction=reduction)
    want = det.policy_loss(lp, old, adv, mask, ref_logprob=ref, **opts)
    count = det.policy_loss_forward(lp, old, adv, mask, ref_logprob=ref, **opts)[1]
    g = torch.ones((), device=DEV)
    dlp = det.policy_loss_backward(g, lp, old, adv, mask, count, ref_logprob=ref, **opts)
    for seed in range(3):
        p = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).to(DEV)
        got = det.policy_loss(lp[p], old[p], adv[p], mask[p], ref_logprob=ref[p], **opts)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # a row's gradient is its own: the same bits with the same divisors
    assert torch.equal(det.policy_loss_backward(g, lp[p], old[p], adv[p], mask[p], torch.cat([count[:-1][p], count[-1:]]),
                                                ref_logprob=ref[p], **opts), dlp[p])


@pytest.mark.parametrize("T", [1, 5, 300, 512])
@pytest.mark.parametrize("B", [1, 16, 17, 32])
def test_a_few_rows_and_the_same_among_others(B, T):
    """Rows that one launch takes, and in a batch whose other rows do not count: the same sums."""
    lp, old, adv, mask, ref = answers(22, B, T, masked=False)
    wide = lambda t, fill: torch.cat([t, torch.full((40, T), fill, device=DEV, dtype=t.dtype)])
    for reduction in ("tokens", "sequences"):
        few, count = det.policy_loss_forward(lp, old, adv, None, ref_logprob=ref, kl_weight=0.1, reduction=reduction)
        all_, many = det.policy_loss_forward(*(wide(t, NAN) for t in (lp, old, adv)),
                                             wide(torch.ones(B, T, device=DEV, dtype=torch.bool), False),
                                             ref_logprob=wide(ref, NAN), kl_weight=0.1, reduction=reduction)
        assert all(torch.equal(a, b) for a, b in zip(few, all_))
        assert torch.equal(count[:B], many[:B]) and count[B] == many[B + 40] and not many[B:B + 40].any()


@pytest.mark.parametrize("reduction", ["tokens", "sequences", "none"])
def test_nothing_that_counts(reduction):
    lp = torch.full((5, 40), NAN, device=DEV, requires_grad=True)
    none = torch.zeros(5, 40, dtype=torch.bool, device=DEV)
    r = det.policy_loss(lp, lp.detach(), lp.detach()[:, 0], none, ref_logprob=lp.detach(), kl_weight=0.5, reduction=reduction)
    assert all((t == 0).all() for t in r)
    g, = torch.autograd.grad(r.loss.sum(), lp)
    assert (g == 0).all()
    for B, T in ((0, 4), (4, 0), (0, 0)):
        lp = torch.zeros(B, T, device=DEV, requires_grad=True)
        r = det.policy_loss(lp, lp.detach(), torch.zeros(B, device=DEV), reduction=reduction)
        assert r.loss.shape == ((B, T) if reduction == "none" else ()) and (r.loss == 0).all()
        assert torch.autograd.grad(r.loss.sum(), lp)[0].shape == (B, T)


def test_values_that_are_not_finite():
    det.device_status()
    zero = torch.zeros(3, 600, device=DEV)
    adv = torch.ones(3, device=DEV)
    masked = torch.ones(3, 600, dtype=torch.bool, device=DEV)
    masked[1, 500] = False
    lp = zero.clone()
    lp[1, 500] = NAN
    assert torch.isfinite(det.policy_loss(lp, zero, adv, masked).loss) and not det.device_status()
    assert torch.isnan(det.policy_loss(lp, zero, adv).loss) and "nonfinite" in det.device_status()
    # a token that the policy rules out: no probability, no gradient; against the reference an infinite estimate
    lp[1, 500] = -INF
    lp.requires_grad_(True)
    r = det.policy_loss(lp, zero, adv, reduction="none")
    g, = torch.autograd.grad(r.loss.sum(), lp)
    assert r.loss[1, 500] == 0 and g[1, 500] == 0 and r.clipped.sum() == 0
    r = det.policy_loss(lp, zero, adv, ref_logprob=zero)
    assert r.kl == INF and r.loss == -1799 / 1800          # reported only
    r = det.policy_loss(lp, zero, adv, ref_logprob=zero, kl_weight=0.1, reduction="sequences")
    assert r.loss == INF and r.kl == INF
    both = zero.clone()
    both[0, 0], both[2, 0] = 200.0, 200.0
    adv = torch.tensor([-1.0, 1.0, -1.0], device=DEV)
    assert det.policy_loss(both, zero, adv).loss == INF    # a negative advantage is not clipped above
    adv[2] = 1.0
    assert det.policy_loss(both, zero, adv).loss == INF    # the other one is
    det.device_status()


def test_small_differences_keep_their_precision():
    # k ~ q^2 / 2 and its slope q, down to the smallest q
    q = torch.tensor([s * 10.0 ** -e for e in range(0, 19) for s in (1.0, -0.7)], dtype=torch.float64)
    lp = torch.zeros(q.numel(), device=DEV, requires_grad=True)
    ref = q.float().to(DEV)
    r = det.policy_loss(lp, lp.detach(), torch.zeros((), device=DEV), ref_logprob=ref, kl_weight=1.0, reduction="none")
    g, = torch.autograd.grad(r.loss.sum(), lp)
    x = ref.double()
    series = sum(x ** k / float(math.factorial(k)) for k in range(2, 25))
    within(r.kl, series, 12 * U * series, "kl")
    rise = torch.expm1(x)
    within(g, -rise, 8 * U * rise.abs(), "slope")


def test_policy_layouts():
    B, T = 6, 70
    lp, old, adv, mask, ref = answers(3, B, T)
    want = det.policy_loss(lp, old, adv, mask, ref_logprob=ref, kl_weight=0.2, reduction="none")
    def odd(t):
        r = torch.zeros(B, T + 5, device=DEV, dtype=t.dtype)
        r[:, 3:-2] = t
        return r[:, 3:-2]
    turned = lambda t: t.t().contiguous().t()
    shaped = lambda t: t.reshape(2, 3, T)
    for f in (odd, turned, shaped):
        got = det.policy_loss(f(lp), f(old), f(adv), f(mask), ref_logprob=f(ref), kl_weight=0.2, reduction="none")
        assert all(torch.equal(a.reshape(B, T), b) for a, b in zip(got, want))
    for red in ("tokens", "sequences"):
        whole = det.policy_loss(lp, old, adv, mask, reduction=red)
        for f in (odd, turned, shaped):
            assert torch.equal(det.policy_loss(f(lp), f(old), f(adv), f(mask), reduction=red).loss, whole.loss)
    # one value to a row is the row of that value, and an expanded one
    a = adv[:, 0].contiguous()
    one = det.policy_loss(lp, old, a, mask).loss
    assert torch.equal(one, det.policy_loss(lp, old, a[:, None].expand(B, T), mask).loss)
    assert torch.equal(one, det.policy_loss(lp, old, torch.stack([a, a], 1)[:, 0], mask).loss)
    # incoming gradients of any stride
    for g in (torch.randn(B, T, device=DEV), torch.randn(T, B, device=DEV).t(), torch.randn(B, 1, device=DEV).expand(B, T),
              torch.ones((), device=DEV).expand(B, T)):
        x = lp.clone().requires_grad_(True)
        y = det.policy_loss(x, old, adv, mask, ref_logprob=ref, kl_weight=0.2, reduction="none").loss
        d, = torch.autograd.grad(y, x, g)
        e, = torch.autograd.grad(det.policy_loss(x, old, adv, mask, ref_logprob=ref, kl_weight=0.2, reduction="none").loss, x, g.contiguous())
        assert torch.equal(d, e)


def test_policy_gradient_against_differences():
    lp, old, adv, mask, ref = answers(4, 5, 40)
    lp = torch.where(mask, lp, 0.0)
    d = (lp - torch.where(mask, old, 0.0)).double()
    away = ((d - math.log(1.2)).abs() > 0.02) & ((d - math.log(0.8)).abs() > 0.02)     # from the kinks
    lp.requires_grad_(True)
    opts = dict(ref_logprob=ref, kl_weight=0.4, reduction="none")
    y = det.policy_loss(lp, old, adv, mask, **opts).loss
    g, = torch.autograd.grad(y.sum(), lp)
    h = 2.0 ** -7
    with torch.no_grad():
        up, down = (lp + h).detach(), (lp - h).detach()
        slope = (det.policy_loss(up, old, adv, mask, **opts).loss.double() -
                 det.policy_loss(down, old, adv, mask, **opts).loss.double()) / (up.double() - down.double())
        size = torch.where(mask, torch.exp(d) * adv.double().abs() + torch.exp((ref - lp).double()), 0.0)
        # third derivatives h^2 / 6, roundings of the two values over 2 h
        bound = (h * h / 4 + 32 * U / h) * (size + 2.0 + (ref - lp).double().abs().nan_to_num())
    pick = away & mask
    within(g[pick], slope[pick], bound[pick], "differences")


# ---------------------------------------------------------------- preference loss

def pairs(seed, P, Tc, Tr, ref=True, masked=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for T in (Tc, Tr):
        lp = -torch.abs(1.5 * torch.randn(P, T, generator=g, device=DEV))
        mask = None
        if masked:
            mask = torch.rand(P, T, generator=g, device=DEV) < 0.6
            if P > 2:
                mask[P // 2] = False
            lp = lp.masked_fill(~mask, INF)
        out.append((lp, lp + 0.4 * torch.randn(P, T, generator=g, device=DEV) if ref else None, mask))
    return out


def preference64(sides, kind, beta, margin, smooth, by_length):
    s, n = [], []
    for lp, ref, mask in sides:
        d = lp.double() - (0.0 if ref is None else ref.double())
        if mask is not None:
            d = d.masked_fill(~mask, 0.0)
        c = torch.full(d.shape[:1], d.shape[1], device=DEV).double() if mask is None else mask.sum(1).double()
        n.append(c.clamp(min=1) if by_length else torch.ones_like(c))
        s.append(d.sum(1) / n[-1])
    ahead = (s[0] - s[1]).requires_grad_(True)
    z = beta * ahead - margin
    if kind == "sigmoid":
        loss = -(1 - smooth) * torch.nn.functional.logsigmoid(z) - smooth * torch.nn.functional.logsigmoid(-z)
    elif kind == "hinge":
        loss = torch.clamp(1 - z, min=0)
    else:
        loss = (ahead - 0.5 / beta) ** 2
    slope, = torch.autograd.grad(loss.sum(), ahead)
    return loss.detach(), beta * s[0], beta * s[1], slope / n[0], -slope / n[1]


@pytest.mark.parametrize("kind,margin,smooth,by_length", [("sigmoid", 0.0, 0.0, False), ("sigmoid", 0.3, 0.2, True),
                                                          ("hinge", -0.1, 0.0, False), ("ipo", 0.0, 0.0, True)])
@pytest.mark.parametrize("P,Tc,Tr,ref,masked", [(1, 1, 1, True, False), (3, 7, 30, True, True), (16, 128, 150, False, True),
                                                (5, 512, 2048, True, True), (4, 2049, 3, True, True), (2, 20000, 9001, False, False),
                                                (900, 5, 6, True, True)])
def test_preference_against_64_bits(P, Tc, Tr, ref, masked, kind, margin, smooth, by_length):
    announce(f"preference {P} {Tc} {Tr} {ref} {masked} {kind}")
    sides = pairs(5, P, Tc, Tr, ref, masked)
    beta = 0.15
    want = preference64(sides, kind, beta, margin, smooth, by_length)
    (c, rc, mc), (r, rr, mr) = sides
    opts = dict(chosen_mask=mc, rejected_mask=mr, kind=kind, beta=beta, margin=margin, label_smoothing=smooth, by_length=by_length)
    c.requires_grad_(True)
    r.requires_grad_(True)
    got = det.preference_loss(c, r, rc, rr, **opts)
    # 64 bits until the last rounding; sums of up to 2^15 differences of size 2^6 lose 2^-30 at most
    for name, a, b in zip(("loss", "chosen", "rejected"), got, want):
        assert a.shape == (P,)
        within(a.detach(), b, 1.01 * U * b.abs() + 2.0 ** -30, name)
    g = torch.rand(P, device=DEV) + 0.5
    dc, dr = torch.autograd.grad(got.loss, (c, r), g)
    for name, d, s, m, T in (("dchosen", dc, want[3], mc, Tc), ("drejected", dr, want[4], mr, Tr)):
        full = (s * g.double())[:, None].expand(P, T)
        if m is not None:
            full = full.masked_fill(~m, 0.0)
            assert (d[~m] == 0).all()
        within(d, full, 2.02 * U * full.abs() + 2.0 ** -30, name)
    f, slope = det.preference_loss_forward(c.detach(), r.detach(), rc, rr, **opts)
    assert all(torch.equal(a.detach(), b) for a, b in zip(got, f))
    both = det.preference_loss_backward(g, slope, c.shape, r.shape, chosen_mask=mc, rejected_mask=mr)
    assert torch.equal(both[0], dc) and torch.equal(both[1], dr)
    # one side alone; one value for every pair
    only, = torch.autograd.grad(det.preference_loss(c.detach(), r, rc, rr, **opts).loss.sum(), r)
    ones = det.preference_loss_backward(torch.ones((), device=DEV).expand(P), slope, c.shape, r.shape, chosen_mask=mc, rejected_mask=mr)
    assert torch.equal(only, ones[1])


def test_a_pair_is_the_same_in_any_batch_and_layout():
    (c, rc, mc), (r, rr, mr) = pairs(6, 50, 700, 33)
    want = det.preference_loss(c, r, rc, rr, chosen_mask=mc, rejected_mask=mr)
    for s in (slice(0, 1), slice(20, 31), slice(49, 50)):
        got = det.preference_loss(c[s], r[s], rc[s], rr[s], chosen_mask=mc[s], rejected_mask=mr[s])
        assert all(torch.equal(a, b[s]) for a, b in zip(got, want))
    turned = lambda t: t.t().contiguous().t()
    got = det.preference_loss(turned(c), r.reshape(5, 10, 33).reshape(50, 33), turned(rc), turned(rr), chosen_mask=turned(mc), rejected_mask=mr)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = det.preference_loss(*(t.reshape(5, 10, -1) for t in (c, r, rc, rr)), chosen_mask=mc.reshape(5, 10, -1),
                              rejected_mask=mr.reshape(5, 10, -1))
    assert all(torch.equal(a.reshape(50), b) for a, b in zip(got, want))


def test_preference_limits():
    det.device_status()
    c = torch.tensor([[1e4], [-1e4], [0.0]], device=DEV, requires_grad=True)
    r = torch.zeros(3, 0, device=DEV, requires_grad=True)          # an answer without a token
    got = det.preference_loss(c, r, beta=1.0)
    g, h = torch.autograd.grad(got.loss.sum(), (c, r))
    assert got.loss.tolist() == [0.0, 1e4, pytest.approx(math.log(2), rel=2 * U)]
    assert g.flatten().tolist() == [0.0, -1.0, -0.5] and h.shape == (3, 0)
    assert got.rejected_reward.tolist() == [0.0, 0.0, 0.0] and not det.device_status()
    bad = torch.tensor([[INF], [NAN], [0.0]], device=DEV)
    for kind in ("sigmoid", "hinge", "ipo"):
        y = det.preference_loss(bad, torch.zeros(3, 1, device=DEV), kind=kind).loss
        assert torch.isnan(y[1]) and torch.isfinite(y[2]) and y[0] == (INF if kind == "ipo" else 0.0)
        assert "nonfinite" in det.device_status()
    empty = det.preference_loss(torch.zeros(0, 4, device=DEV), torch.zeros(0, 5, device=DEV))
    assert all(t.shape == (0,) for t in empty)


# ---------------------------------------------------------------- together

def test_with_the_scores_that_feed_them():
    # a policy step from logits, the gradient of the logits against 64 bits
    B, T, V = 4, 30, 201
    g = torch.Generator(device=DEV).manual_seed(7)
    z = (2.0 * torch.randn(B, T, V, generator=g, device=DEV)).requires_grad_(True)
    t = torch.randint(0, V, (B, T), generator=g, device=DEV)
    mask = torch.rand(B, T, generator=g, device=DEV) < 0.8
    old = torch.log_softmax(z.detach(), -1).gather(-1, t[..., None])[..., 0] + 0.2 * torch.randn(B, T, generator=g, device=DEV)
    ref = old + 0.1
    adv = torch.randn(B, generator=g, device=DEV)
    loss = det.policy_loss(det.token_logprobs(z, t).logprob, old, adv, mask, ref_logprob=ref, kl_weight=0.1).loss
    dz, = torch.autograd.grad(loss, z)
    Z = z.detach().double().requires_grad_(True)
    lp = torch.log_softmax(Z, -1).gather(-1, t[..., None])[..., 0]
    r, q = torch.exp(lp - old.double()), ref.double() - lp
    a = adv.double()[:, None]
    l = -torch.minimum(r * a, r.clamp(0.8, 1.2) * a) + 0.1 * (torch.exp(q) - 1 - q)
    want = (l * mask).sum() / mask.sum()
    dZ, = torch.autograd.grad(want, Z)
    assert abs(loss.item() - want.item()) <= 2.0 ** -18
    # the log probability is off by a few half steps of its terms (size 2^4), which the ratio and the weights carry
    assert (dz.double() - dZ).abs().max() <= 2.0 ** -16 * dZ.abs().max()


def test_streams_and_graphs():
    def step(lp, old, adv, mask, ref, c, r, mc, mr):
        out = []
        for red in ("tokens", "sequences", "none"):
            p, count = det.policy_loss_forward(lp, old, adv, mask, ref_logprob=ref, kl_weight=0.1, reduction=red)
            g = torch.ones_like(p.loss)
            out += [*p, det.policy_loss_backward(g, lp, old, adv, mask, count, ref_logprob=ref, kl_weight=0.1, reduction=red)]
        q, slope = det.preference_loss_forward(c, r, chosen_mask=mc, rejected_mask=mr)
        return [*out, *q, *det.preference_loss_backward(torch.ones_like(q.loss), slope, c.shape, r.shape, chosen_mask=mc, rejected_mask=mr)]

    def data(seed):
        a = answers(seed, 3000, 9)
        (c, _, mc), (r, _, mr) = pairs(seed, 20, 600, 5)
        return [*a, c, r, mc, mr]
    args = data(8)
    want = step(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    bufs = [t.clone() for t in args]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*bufs)
    for k in range(3):
        for b, t in zip(bufs, data(9 + k)):
            b.copy_(t)
        graph.replay()
        eager = step(*bufs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_second_derivatives_are_refused():
    lp, old, adv, mask, _ = answers(10, 4, 20, ref=False)
    x = torch.where(mask, lp, 0.0).requires_grad_(True)
    g, = torch.autograd.grad(det.policy_loss(x, old, adv, mask).loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(g.square().sum(), x)
    for i in range(2):
        c = [torch.randn(4, 6, device=DEV, requires_grad=j == i) for j in range(2)]
        g, = torch.autograd.grad(det.preference_loss(*c).loss.sum(), c[i], create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            torch.autograd.grad(g.square().sum(), c[i])


def test_other_inputs_are_constants():
    lp, old, adv, mask, ref = (t if t is None or t.dtype == torch.bool else torch.nan_to_num(t).requires_grad_(True)
                               for t in answers(11, 4, 20))
    r = det.policy_loss(lp, old, adv, mask, ref_logprob=ref, kl_weight=0.1)
    assert not r.kl.requires_grad and not r.clipped.requires_grad
    grads = torch.autograd.grad(r.loss, (lp, old, adv, ref), allow_unused=True)
    assert grads[0] is not None and grads[1:] == (None, None, None)
    assert not det.policy_loss(lp.detach(), old, adv, mask).loss.requires_grad


def test_rows_past_32_bits():
    # offsets of the last rows pass 2^32 bytes; masks' pass 2^31
    B, T = 140000, 8192
    lp = torch.zeros(B, T, device=DEV)
    mask = torch.zeros(B, T, dtype=torch.bool, device=DEV)
    lp[-1, -3:] = torch.tensor([0.1, -0.2, 0.05], device=DEV)
    mask[-1, -3:] = True
    old, adv = torch.zeros((), device=DEV).expand(B, T), torch.ones((), device=DEV).expand(B)
    p, count = det.policy_loss_forward(lp, old, adv, mask)
    small, c2 = det.policy_loss_forward(lp[-1:], old[-1:], adv[-1:], mask[-1:])
    assert all(torch.equal(a, b) for a, b in zip(p, small)) and count[-1] == 3
    one = torch.ones((), device=DEV)
    d = det.policy_loss_backward(one, lp, old, adv, mask, count)
    assert torch.equal(d[-1:], det.policy_loss_backward(one, lp[-1:], old[-1:], adv[-1:], mask[-1:], c2)) and (d[:-1] == 0).all()


def test_rows_that_cancel_are_added_exactly():
    # with r = 1 a token's loss is -A, exactly; a row of two has a sum of at most 48 bits
    g = torch.Generator().manual_seed(12)
    for B, T in ((5000, 1), (20001, 2)):
        adv = torch.randn(B, T, generator=g) * torch.exp(2 * torch.randn(B, 1, generator=g))
        adv[B // 2:2 * (B // 2)] = -adv[:B // 2]                  # what is left is the last row, and a trace
        adv[3, 0] += 2.0 ** -20
        lp = -torch.rand(B, T, generator=g)
        total = torch.tensor(math.fsum((-adv.double()).flatten().tolist()), dtype=torch.float64).float()
        want = (total.double() / (B * T)).float()
        got = det.policy_loss(lp.to(DEV), lp.to(DEV), adv.to(DEV)).loss
        assert got.item() == want.item()
