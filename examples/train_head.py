"""Train a small language-model head bit-reproducibly, then read it.

A student (DetLayerNorm -> DetLinear -> DetLayerNorm -> DetLinear onto the
vocabulary) learns next tokens from a fixed teacher: per step the mean, formed
exactly, of the distillation loss against the teacher's top logits and of the
given tokens' negative log probability.  Afterwards it scores a held-out batch
and decodes greedily, one token at a time.

    python examples/train_head.py [--steps 40] [--vocab 5003] [--width 256] [--tokens 512]

It trains twice and shows that every loss and every weight has the same bits,
and that the norm's weight gradient of two row shards, added in the long
accumulator, is the unsharded one.
"""
from __future__ import annotations

import argparse
import hashlib
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitwise_deterministic_exact_amd as det  # noqa: E402


class Head(torch.nn.Module):
    """[..., width] hidden states -> [..., vocab] float32 logits."""

    def __init__(self, width: int, vocab: int, device):
        super().__init__()
        bf16 = torch.bfloat16
        self.norm1 = det.DetLayerNorm(width, device=device, dtype=bf16, out_dtype=bf16)
        self.mix = det.DetLinear(width, width, device=device, dtype=bf16)
        self.norm2 = det.DetLayerNorm(width, device=device, dtype=bf16, out_dtype=bf16)
        self.out = det.DetLinear(width, vocab, device=device, dtype=bf16)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return self.out(self.norm2(self.mix(self.norm1(x))))


def make_data(width: int, vocab: int, tokens: int, top: int, device):
    """Token embeddings, a batch of (token, next token) and a teacher's top logits for it."""
    g = torch.Generator().manual_seed(11)
    embed = torch.randn(vocab, width, generator=g).to(device)
    succ = torch.randperm(vocab, generator=g).to(device)          # the language: each token has one successor
    token = torch.randint(0, min(vocab, 4 * width), (tokens,), generator=g).to(device)
    index = torch.stack([torch.randint(0, vocab, (top - 1,), generator=g) for _ in range(tokens)]).to(device)
    index = torch.cat([succ[token][:, None], index], dim=1)
    teacher = torch.cat([torch.full((tokens, 1), 8.0), 2.0 * torch.rand(tokens, top - 1, generator=g)], dim=1)
    return embed, succ, token, teacher.to(device), index


def train(steps: int, width: int, vocab: int, tokens: int, top: int = 16, temperature: float = 2.0, lr: float = 4.0,
          device="cuda:0"):
    """(head, losses, digest): digest is SHA-256 over every loss and final weight."""
    torch.manual_seed(5)
    head = Head(width, vocab, device)
    embed, succ, token, teacher, index = make_data(width, vocab, tokens, top, device)
    master = [p.detach().float().clone() for p in head.parameters()]
    losses = []
    for _ in range(steps):
        logits = head(embed[token])
        kl = det.exact_mean(det.distill_loss(logits, teacher, index, temperature=temperature))
        scored = det.token_logprobs(logits, succ[token])
        loss = kl - det.exact_mean(scored.logprob)
        grads = torch.autograd.grad(loss, list(head.parameters()))
        with torch.no_grad():
            for p, m, g in zip(head.parameters(), master, grads):
                m -= lr * g.float()
                p.copy_(m.to(p.dtype))
        losses.append(loss.detach())
    losses = torch.stack(losses)
    h = hashlib.sha256(losses.cpu().numpy().tobytes())
    for p in head.parameters():
        h.update(p.detach().cpu().view(torch.int16).numpy().tobytes())
    return head, losses, h.hexdigest()


@torch.no_grad()
def score(head: Head, embed: torch.Tensor, token: torch.Tensor, target: torch.Tensor, top: int = 5):
    """Log probabilities of the targets, entropies and alternatives."""
    return det.token_logprobs(head(embed[token]), target, top=top)


@torch.no_grad()
def decode(head: Head, embed: torch.Tensor, first: int, length: int):
    """Greedy continuation, one token at a time: [(token, its log probability)]."""
    out, token = [], torch.tensor([first], device=embed.device)
    for _ in range(length):
        r = det.token_logprobs(head(embed[token]), top=1)
        token = r.top_index[:, 0]
        out.append((token, r.top_logprob[:, 0]))
    return [(int(t), float(p)) for t, p in out]


def shard_check(head: Head, embed: torch.Tensor, token: torch.Tensor) -> bool:
    """norm1's weight gradient over two row shards, as ranks of a data-parallel
    job would compute it: the raw digits added, rounded once."""
    x = embed[token]
    _, mean, rstd = det.layer_norm_forward(x, head.norm1.weight, head.norm1.bias)
    g = torch.Generator().manual_seed(3)
    dy = torch.randn(x.shape, generator=g).to(x.device)
    whole = det.layer_norm_backward(dy, x, None, mean, rstd)
    cut = x.shape[0] // 2 // det.NORM_SHARD_ROWS * det.NORM_SHARD_ROWS
    parts = [det.layer_norm_digits(dy[s], x[s], mean[s], rstd[s]) for s in (slice(0, cut), slice(cut, None))]
    dw, db = det.det_finalize(det.det_combine(parts))
    return torch.equal(dw, whole[1]) and torch.equal(db, whole[2])


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args(argv)
    head, losses, digest = train(a.steps, a.width, a.vocab, a.tokens)
    _, _, again = train(a.steps, a.width, a.vocab, a.tokens)
    embed, succ, token, _, _ = make_data(a.width, a.vocab, a.tokens, 16, "cuda:0")
    r = score(head, embed, token, succ[token])
    first = int(token[0])
    walk = decode(head, embed, first, 4)
    result = {
        "first_loss": float(losses[0]), "last_loss": float(losses[-1]), "digest": digest, "repeats": digest == again,
        "shards_agree": shard_check(head, embed, token), "mean_logprob": float(det.exact_mean(r.logprob)),
        "mean_entropy": float(det.exact_mean(r.entropy)),
        "top1_accuracy": float((r.top_index[:, 0] == succ[token]).float().mean()), "decoded": walk,
    }
    for k, v in result.items():
        print(f"{k}: {v}", flush=True)
    return result


if __name__ == "__main__":
    main()
