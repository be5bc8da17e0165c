"""Layer norm, token log probabilities and distillation under torch's other
transforms (CPU: each is refused before the device is looked at)."""
import pytest
import torch
import torch.autograd.forward_ad as fw
from torch.fx.experimental.proxy_tensor import make_fx

import bitwise_deterministic_exact_amd as det


def _m(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


T, INDEX = _m(2, dtype=torch.int64), _m(2, 3, dtype=torch.int64)
CALLS = {
    "layer_norm": lambda x: det.layer_norm(x),
    "layer_norm of the weight": lambda x: det.layer_norm(_m(2, 8), x[0]),
    "layer_norm of the bias": lambda x: det.layer_norm(_m(2, 8), None, x[0]),
    "DetLayerNorm": lambda x: det.DetLayerNorm(8, device="meta")(x),
    "token_logprobs": lambda x: det.token_logprobs(x, T).logprob,
    "alternatives": lambda x: det.token_logprobs(x, top=2).top_logprob,
    "distill_loss": lambda x: det.distill_loss(x, _m(2, 3), INDEX),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_forward_mode_is_refused(name):
    with fw.dual_level():
        for x in (fw.make_dual(_m(2, 8), _m(2, 8)), fw.make_dual(_m(2, 8).requires_grad_(True), _m(2, 8))):
            with pytest.raises(RuntimeError, match="forward-mode"):
                CALLS[name](x)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
                CALLS[name](x)                     # no_grad is about the reverse mode
        with fw._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="GPU"):
            CALLS[name](fw.make_dual(_m(2, 8), _m(2, 8)))


def _traced_calls():
    c = torch.zeros
    i2, i3 = c(2, dtype=torch.int64), c(2, 3, dtype=torch.int64)
    return {
        "layer_norm": lambda x: det.layer_norm(x),
        "layer_norm_forward": lambda x: det.layer_norm_forward(x)[0],
        "layer_norm_backward": lambda x: det.layer_norm_backward(x, x, None, c(2), c(2))[0],
        "layer_norm_digits": lambda x: det.layer_norm_digits(x, x, c(2), c(2)),
        "token_logprobs": lambda x: det.token_logprobs(x, i2).logprob,
        "token_logprobs_forward": lambda x: det.token_logprobs_forward(x, i2)[1],
        "token_logprobs_backward": lambda x: det.token_logprobs_backward(x, i2, c(2, 4), g_logprob=c(2)),
        "distill_loss": lambda x: det.distill_loss(x, c(2, 3), i3),
        "distill_forward": lambda x: det.distill_forward(x, c(2, 3), i3)[0],
        "distill_backward": lambda x: det.distill_backward(x, i3, c(2, 4), c(2, 3), c(2)),
        "exact_mean": lambda x: det.exact_mean(x),
    }


@pytest.mark.parametrize("name", list(_traced_calls()))
def test_traces_are_refused(name):
    # a trace would record the results' allocation and nothing that fills it
    call, x = _traced_calls()[name], torch.randn(2, 8)
    with pytest.raises(RuntimeError, match="cannot be traced"):
        torch.jit.trace(call, (x,), check_trace=False)
    for mode in ({}, {"pre_dispatch": True}, {"tracing_mode": "fake", "_allow_non_fake_inputs": True}):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(call, **mode)(x)
    with pytest.raises(Exception) as e:            # an untraced call gets as far as the device
        call(x)
    assert "traced" not in str(e.value)
