"""What layer norm, token log probabilities and distillation say to requests
for derivatives that they do not form: an error, never a result that leaves
terms out."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import bitwise_deterministic_exact_amd as det

pytestmark = pytest.mark.gpu


def _randn(*shape, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def _ops():
    """name: (call of the leaf, shape of the leaf)"""
    w, b = 1 + 0.1 * _randn(20, seed=2), _randn(20, seed=3)
    t = torch.arange(3, device="cuda")
    teacher, index = _randn(3, 4, seed=4), torch.arange(12, device="cuda").reshape(3, 4)
    return {
        "layer_norm of x": (lambda x: det.layer_norm(x, w, b), (3, 20)),
        "layer_norm of the weight": (lambda v: det.layer_norm(_randn(3, 20, seed=5), v, b), (20,)),
        "layer_norm of the bias": (lambda v: det.layer_norm(_randn(3, 20, seed=5), w, v), (20,)),
        "token_logprobs": (lambda z: det.token_logprobs(z, t).logprob, (3, 20)),
        "entropy": (lambda z: det.token_logprobs(z).entropy, (3, 20)),
        "alternatives": (lambda z: det.token_logprobs(z, top=3).top_logprob, (3, 20)),
        "distill_loss": (lambda z: det.distill_loss(z, teacher, index, temperature=2.0), (3, 20)),
    }


@pytest.mark.parametrize("name", ["layer_norm of x", "layer_norm of the weight", "token_logprobs", "entropy",
                                  "alternatives", "distill_loss"])
def test_derivatives_of_gradients_are_refused(name):
    # the incoming gradient is a constant, as for any loss that is linear in the result
    call, shape = _ops()[name]
    leaf = _randn(*shape, seed=6).requires_grad_(True)
    first, = torch.autograd.grad(call(leaf).sum(), leaf)
    assert not first.requires_grad
    g, = torch.autograd.grad(call(leaf).sum(), leaf, create_graph=True)
    assert g.requires_grad and torch.equal(g.detach(), first)
    penalty = g.pow(2).sum()
    refused = pytest.raises(RuntimeError, match="differentiable once")
    with refused:
        torch.autograd.grad(penalty, leaf, retain_graph=True)
    with refused:                                  # nor are the first-order terms passed off as the whole
        torch.autograd.grad(call(leaf).sum() + penalty, leaf, retain_graph=True)
    with refused:
        torch.autograd.grad(penalty, leaf, retain_graph=True, allow_unused=True)
    with refused:
        (call(leaf).sum() + penalty).backward()


def test_derivatives_in_the_incoming_gradient_are_refused():
    for call, shape in _ops().values():
        leaf = _randn(*shape, seed=6).requires_grad_(True)
        scale = torch.ones((), device="cuda", requires_grad=True)
        g, = torch.autograd.grad(call(leaf).sum() * scale, leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            torch.autograd.grad(g.sum(), scale)


def test_tangents_of_incoming_gradients_are_refused():
    for call, shape in _ops().values():
        leaf = _randn(*shape, seed=6).requires_grad_(True)
        y = call(leaf)
        with fw.dual_level():
            dual = fw.make_dual(torch.ones_like(y), torch.ones_like(y))
            with pytest.raises(RuntimeError, match="forward-mode"):
                torch.autograd.grad(y, leaf, dual)


def test_exact_mean_takes_the_derivatives_it_can():
    t = _randn(7, seed=8).requires_grad_(True)
    g, = torch.autograd.grad(det.exact_mean(t * t), t, create_graph=True)
    h, = torch.autograd.grad(g.sum(), t)           # of 2 t / 7
    want = torch.full((7,), 2.0, device="cuda") * (torch.ones((), device="cuda") / torch.full((), 7.0, device="cuda"))
    assert torch.equal(h, want)
    with fw.dual_level(), pytest.raises(RuntimeError):
        det.exact_mean(fw.make_dual(_randn(7), _randn(7)))
