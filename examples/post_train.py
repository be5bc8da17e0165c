"""Post-train a small feed-forward language model bit-reproducibly.

A model (embedding -> norm -> gated projection -> DetLinear -> norm -> DetLinear
onto the vocabulary, its activations kept in 8 bits between the passes) first
samples answers, is scored by a fixed reward (even tokens are good), and takes
steps on the clipped policy loss with a KL term towards the model it started
from; then it takes steps on the preference loss over pairs of the same answers.

    python examples/post_train.py [--steps 6] [--width 128] [--hidden 320] [--vocab 501] [--answers 12] [--length 24]

It runs twice and shows that every loss and every weight has the same bits, and
that an answer's log probabilities are the same alone and in the batch.
"""
from __future__ import annotations

import argparse
import hashlib
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_deterministic_exact_amd as det  # noqa: E402

BF16 = torch.bfloat16


class Model(torch.nn.Module):
    """[...] tokens -> [..., vocab] float32 logits of the next one."""

    def __init__(self, vocab: int, width: int, hidden: int, device, checkpoint="int8"):
        super().__init__()
        g = torch.Generator().manual_seed(3)
        self.register_buffer("embed", torch.randn(vocab, width, generator=g).to(device))
        self.norm1 = det.DetLayerNorm(width, device=device, dtype=BF16, out_dtype=BF16)
        self.up = det.DetGatedLinear(width, hidden, device=device, checkpoint=checkpoint)
        self.down = det.DetLinear(hidden, width, device=device, dtype=BF16, checkpoint=checkpoint)
        self.norm2 = det.DetLayerNorm(width, device=device, dtype=BF16, out_dtype=BF16)
        self.head = det.DetLinear(width, vocab, device=device, dtype=BF16)

    def forward(self, token: torch.Tensor) -> torch.Tensor:
        x = self.embed[token]
        x = x + self.down(self.up(self.norm1(x)))
        return self.head(self.norm2(x))


@torch.no_grad()
def sample(model: Model, first: torch.Tensor, length: int, seed: int) -> torch.Tensor:
    """Answers of `length` tokens after each of `first`, one token at a time: [answers, length + 1]."""
    g = torch.Generator().manual_seed(seed)
    out = [first]
    for _ in range(length):
        noise = -torch.log(-torch.log(torch.rand(first.numel(), model.embed.shape[0], generator=g))).to(first.device)
        out.append(det.token_logprobs(model(out[-1]) + noise, top=1).top_index[:, 0])
    return torch.stack(out, dim=1)


def logprobs(model: Model, answers: torch.Tensor) -> torch.Tensor:
    """Log probability of each token of the answers but the first: [answers, length]."""
    return det.token_logprobs(model(answers[:, :-1]), answers[:, 1:]).logprob


def policy_step_loss(model, answers, old, ref, advantage, mask):
    """The clipped policy loss of the answers, a KL term towards the reference."""
    return det.policy_loss(logprobs(model, answers), old, advantage, mask, ref_logprob=ref, kl_weight=0.05,
                           reduction="sequences")


def preference_step_loss(model, good, bad, ref_good, ref_bad, mask_good, mask_bad):
    """The mean, formed exactly, of the preference loss over pairs of answers."""
    r = det.preference_loss(logprobs(model, good), logprobs(model, bad), ref_good, ref_bad, chosen_mask=mask_good,
                            rejected_mask=mask_bad)
    return det.exact_mean(r.loss)


def post_train(steps: int, width: int, hidden: int, vocab: int, answers: int, length: int, lr: float = 0.5,
               device="cuda:0"):
    """(model, losses, digest): digest is SHA-256 over every loss and final weight."""
    torch.manual_seed(5)
    model = Model(vocab, width, hidden, device)
    first = torch.arange(answers, device=device) % vocab
    tokens = sample(model, first, length, seed=7)
    with torch.no_grad():
        old = logprobs(model, tokens)
    # answers end at different lengths; what follows does not count
    ends = length - torch.arange(answers, device=device) % max(1, length // 2)
    mask = torch.arange(length, device=device) < ends[:, None]
    reward = (((tokens[:, 1:] % 2 == 0) & mask).sum(dim=1) / ends).float()
    advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
    order = reward.argsort(stable=True)
    half = answers // 2
    bad, good = order[:half], order[-half:]
    master = [p.detach().float().clone() for p in model.parameters()]
    losses = []
    for k in range(2 * steps):
        if k < steps:
            loss = policy_step_loss(model, tokens, old, old, advantage, mask).loss
        else:
            loss = preference_step_loss(model, tokens[good], tokens[bad], old[good], old[bad], mask[good], mask[bad])
        grads = torch.autograd.grad(loss, list(model.parameters()))
        with torch.no_grad():
            for p, m, g in zip(model.parameters(), master, grads):
                m -= lr * g.float()
                p.copy_(m.to(p.dtype))
        losses.append(loss.detach())
    losses = torch.stack(losses)
    h = hashlib.sha256(losses.cpu().numpy().tobytes())
    for p in model.parameters():
        h.update(p.detach().cpu().view(torch.int16).numpy().tobytes())
    return model, tokens, losses, h.hexdigest()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=6)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--hidden", type=int, default=320)
    ap.add_argument("--vocab", type=int, default=501)
    ap.add_argument("--answers", type=int, default=12)
    ap.add_argument("--length", type=int, default=24)
    a = ap.parse_args(argv)
    sizes = (a.steps, a.width, a.hidden, a.vocab, a.answers, a.length)
    model, tokens, losses, digest = post_train(*sizes)
    again = post_train(*sizes)[3]
    with torch.no_grad():
        whole = logprobs(model, tokens)
        alone = all(torch.equal(logprobs(model, tokens[i:i + 1])[0], whole[i]) for i in range(min(4, a.answers)))
    result = {"losses": [float(l) for l in losses], "digest": digest, "repeats": digest == again, "alone": alone}
    for k, v in result.items():
        print(f"{k}: {v}", flush=True)
    return result


if __name__ == "__main__":
    main()
