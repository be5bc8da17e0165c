"""The policy and preference losses where fp32 on the way would show: sums and
ratios past its range, one rounding of a mean, differences that it does not
hold, and what a preference loss keeps for its gradient."""
from fractions import Fraction

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24                                      # half a step of fp32


def within(got, want, bound, what):
    assert got.dtype == torch.float32
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off: {got[bad][:3]} for {want[bad][:3]}"


# one launch of few rows, rows of several workgroups, more pieces than one thread adds, several workgroups that join
@pytest.mark.parametrize("reduction", ["tokens", "sequences"])
@pytest.mark.parametrize("B,T", [(1, 4), (20, 300), (40, 7), (3, 5000), (1, 70000), (17000, 3)])
def test_means_whose_sums_pass_fp32(B, T, reduction):
    announce(f"policy far sums {B} {T} {reduction}")
    det.device_status()
    g = torch.Generator(device=DEV).manual_seed(1)
    old = -88.0 - 0.7 * torch.rand(B, T, generator=g, device=DEV)
    lp = torch.zeros(B, T, device=DEV, requires_grad=True)
    adv = torch.full((B,), -1.0, device=DEV)        # a negative advantage is not clipped above: l = e^d up to 3.3e38
    ref = -old
    each, rise = torch.exp(-old.double()), torch.exp(ref.double())
    r = det.policy_loss(lp, old, adv, ref_logprob=ref, reduction=reduction)
    # 8 half steps of a token's value, half a step of the mean
    within(r.loss, each.mean(), 9 * U * each.mean(), "loss")
    kl = (rise - 1 - ref.double()).mean()
    within(r.kl, kl, 9 * U * kl, "kl")
    assert not det.device_status()
    grad, = torch.autograd.grad(r.loss, lp)
    within(grad, each / (B * T), 10 * U * each / (B * T), "gradient")
    # pairs of rows that cancel leave the last one, if any: with r = 1 a token's loss is -A
    adv = torch.where(torch.arange(B, device=DEV) % 2 == 0, -1.0, 1.0) * 2.0 ** 127
    want = 2.0 ** 127 / B if B % 2 else 0.0
    assert det.policy_loss(old, old, adv, reduction=reduction).loss.item() == torch.tensor(want).item()


@pytest.mark.parametrize("reduction", ["tokens", "sequences"])
def test_a_mean_is_rounded_once(reduction):
    """With r = 1 a token's loss is -A, so a mean is a quotient of exact numbers."""
    for seed in range(40):
        g = torch.Generator().manual_seed(seed)
        B, T = (7, 3) if seed % 2 == 0 else (41, 11)
        lp, adv = -torch.rand(B, T, generator=g), torch.randn(B, T, generator=g)
        total = sum(Fraction(v) for v in (-adv.double()).flatten().tolist())
        want = torch.tensor(float(total / (B * T)), dtype=torch.float64).float()
        got = det.policy_loss(lp.to(DEV), lp.to(DEV), adv.to(DEV), reduction=reduction).loss
        assert got.item() == want.item(), seed


def test_ratios_past_fp32():
    """r alone leaves fp32 on either side, r A does not: also where the old policy ruled a token out."""
    low = torch.finfo(torch.float32).min
    d, a = [], []
    for x, y in ((88.9, -1e-10), (100.25, -1e-20), (150.5, -3e-38), (180.125, -2e-45), (-88.5, 1e10), (-100.25, 1e30), (-120.0, 2e38),
                 (-180.0, 3e38), (80.5, -1.0), (-80.5, 1.0), (85.0, -1e-5), (81.0, -1e-44)):
        d.append(x)
        a.append(y)
    # differences that fp32 holds, and some that it does not
    for first in (0.0, -0.7331, -13.37):
        lp = torch.full((len(d),), first, device=DEV, requires_grad=True)
        old, adv = first - torch.tensor(d, device=DEV), torch.tensor(a, device=DEV)
        r = det.policy_loss(lp, old, adv, reduction="none")
        want = -torch.exp(lp.detach().double() - old.double()) * adv.double()
        # four factors (2 units of the exponential, its low part) and four products; below 2^-126 half a step is 2^-150
        within(r.loss, want, 24 * U * want.abs() + 2.0 ** -149, "loss")
        grad, = torch.autograd.grad(r.loss.sum(), lp)
        within(grad, want, 24 * U * want.abs() + 2.0 ** -149, "gradient")
    # no advantage: no loss and no gradient, however far the ratio is
    det.device_status()
    old = torch.tensor([low, -1e9, -89.0, -1000.0, 0.0, 89.0, 1e9, -low], device=DEV)
    lp = torch.zeros(8, device=DEV, requires_grad=True)
    for reduction in ("none", "tokens", "sequences"):
        r = det.policy_loss(lp, old, torch.zeros(8, device=DEV), reduction=reduction)
        grad, = torch.autograd.grad(r.loss.sum(), lp)
        assert (r.loss == 0).all() and (grad == 0).all() and (r.clipped == 0).all()
    assert not det.device_status()
    # with one: clipped, or past fp32
    assert det.policy_loss(lp, old, torch.ones(8, device=DEV), reduction="none").loss.tolist()[:4] == [-torch.tensor(1.2).item()] * 4
    assert (det.policy_loss(lp, old, -torch.ones(8, device=DEV), reduction="none").loss[:2] == float("inf")).all()
    det.device_status()


def test_estimates_of_far_differences():
    """q = ref - logprob needs more than 32 bits: e^q shows what is missing |q| times over."""
    g = torch.Generator(device=DEV).manual_seed(3)
    lp = (-85.0 * torch.rand(4, 3000, generator=g, device=DEV)).requires_grad_(True)
    ref = -85.0 * torch.rand(4, 3000, generator=g, device=DEV)
    r = det.policy_loss(lp, lp.detach(), torch.zeros(4, device=DEV), ref_logprob=ref, kl_weight=1.0, reduction="none")
    grad, = torch.autograd.grad(r.loss.sum(), lp)
    q = ref.double() - lp.detach().double()
    size = torch.exp(q) + 1 + q.abs()
    # e^q: 2 units of the exponential, the low part and its product; two differences: 8 half steps in all
    # (kl: up to |q| = 1 a series, 12 of its own; the gradient's parts there are at most 1)
    within(r.kl, torch.expm1(q) - q, torch.where(q.abs() <= 1.0, 12 * U * size, 8 * U * size), "kl")
    within(grad, -torch.expm1(q), torch.where(q.abs() <= 1.0, 12 * U * size, 8 * U * size), "gradient")


@pytest.mark.parametrize("T", [4, 600, 1500, 2048, 2050, 9000])
def test_an_answers_reward_does_not_depend_on_the_other_answer(T):
    g = torch.Generator(device=DEV).manual_seed(4)
    # what is left of sums that cancel shows their order
    x = torch.randn(5, T // 2, generator=g, device=DEV) * torch.exp(20 * torch.randn(5, T // 2, generator=g, device=DEV))
    x = x.clamp(-1e30, 1e30)
    x = torch.cat([x, -x], 1)[:, torch.randperm(T, generator=g, device=DEV)]
    other = -torch.rand(5, 30, generator=g, device=DEV)
    wide = torch.zeros(5, 7000, device=DEV)
    wide[:, :30] = other
    mask = torch.arange(7000, device=DEV).expand(5, 7000) < 30
    short, long_ = det.preference_loss(x, other), det.preference_loss(x, wide, rejected_mask=mask)
    assert torch.equal(short.chosen_reward, long_.chosen_reward)
    assert torch.equal(det.preference_loss(other, x).rejected_reward, short.chosen_reward)
    assert torch.equal(det.preference_loss(wide, x, chosen_mask=mask).rejected_reward, short.chosen_reward)


def test_a_preference_loss_keeps_no_log_probabilities():
    g = torch.Generator(device=DEV).manual_seed(5)
    base = [(-torch.rand(6, T, generator=g, device=DEV)).requires_grad_(True) for T in (700, 33)]
    mask = torch.rand(6, 700, generator=g, device=DEV) < 0.5
    want = torch.autograd.grad(det.preference_loss(*base, chosen_mask=mask).loss.sum(), base)
    sizes = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append((t.dtype, t.numel())), t)[1], lambda t: t):
        det.preference_loss(*base, chosen_mask=mask)
    assert sorted(sizes, key=str) == sorted([(torch.float32, 12), (torch.bool, 6 * 700)], key=str)
    # the gradient does not need them: they may change in place
    sides = [t * 1.0 for t in base]
    loss = det.preference_loss(*sides, chosen_mask=mask).loss.sum()
    with torch.no_grad():
        for t in sides:
            t.add_(1.0)
    for a, b in zip(torch.autograd.grad(loss, base), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge"])
def test_far_margins(kind):
    c, r = torch.zeros(3, 4, device=DEV, requires_grad=True), torch.zeros(3, 4, device=DEV)
    for margin in (1e6, 3e7, -2e9):
        y = det.preference_loss(c, r, kind=kind, margin=margin)
        want = max(0.0, margin) if kind == "sigmoid" else max(0.0, 1 + margin)
        within(y.loss, torch.full((3,), want, dtype=torch.float64, device=DEV), U * want, "loss")
        grad, = torch.autograd.grad(y.loss.sum(), c)
        assert (grad == (-torch.tensor(0.1).item() if margin > 0 else 0.0)).all()
