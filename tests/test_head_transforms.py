"""Layer norm, token log probabilities and distillation under torch's other
transforms (CPU: each is refused before the device is looked at)."""
import pytest
import torch
import torch.autograd.forward_ad as fw

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
