"""The head example: training repeats bit for bit, learns, its row shards
agree, and its scores match a 64-bit softmax of its own logits."""
import pytest
import torch

import bitwise_deterministic_exact_amd as det
from examples import train_head

pytestmark = pytest.mark.gpu


def test_example_trains_reproducibly():
    r = train_head.main(["--steps", "25", "--vocab", "1003", "--width", "128", "--tokens", "256"])
    assert r["repeats"] and r["shards_agree"]
    assert r["last_loss"] < 0.6 * r["first_loss"] and r["top1_accuracy"] > 0.5
    assert len(r["decoded"]) == 4 and all(0 <= t < 1003 and p <= 0 for t, p in r["decoded"])


def test_scores_match_the_head_s_logits():
    head, _, _ = train_head.train(2, 64, 301, 96, top=4)
    embed, succ, token, _, _ = train_head.make_data(64, 301, 96, 4, "cuda:0")
    r = train_head.score(head, embed, token, succ[token])
    with torch.no_grad():
        l = torch.log_softmax(head(embed[token]).double(), -1)
    want = l.gather(1, succ[token][:, None])[:, 0]
    assert (r.logprob.double() - want).abs().max() <= 2.0 ** -24 * (96 + want.abs().max().item())
    assert torch.equal(r.top_index[:, 0], l.argmax(-1))


def test_step_under_graph_capture():
    # forward and backward of the whole chain captured once, leaves created for
    # the capture alone; every replay against the eager step
    width, vocab, tokens, top = 64, 301, 96, 4
    torch.manual_seed(1)
    head = train_head.Head(width, vocab, "cuda:0")
    embed, succ, token, teacher, index = train_head.make_data(width, vocab, tokens, top, "cuda:0")

    def step(x, params):
        norm1, mix, norm2, out = head.norm1, head.mix, head.norm2, head.out
        h = det.layer_norm(x, params[0], params[1], norm1.eps, torch.bfloat16)
        logits = out(h) if width == vocab else torch.nn.functional.pad(h.float(), (0, vocab - width), value=-5.0)
        loss = det.distill_loss(logits, teacher, index, temperature=2.0)
        lp = det.token_logprobs(logits, succ[token], top=2)
        return torch.autograd.grad((loss, lp.logprob, lp.entropy), (x, *params),
                                   (g, -g, 0.1 * g))

    g = torch.full((tokens,), 1.0 / tokens, device="cuda")
    fresh = lambda: [t.detach().clone().requires_grad_(True)                       # noqa: E731
                     for t in (embed[token], head.norm1.weight, head.norm1.bias)]
    x, w, b = fresh()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(x, (w, b))
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, (w, b))
    for k in range(4):
        with torch.no_grad():
            x.copy_(embed[token] * (0.5 + k))
        graph.replay()
        torch.cuda.synchronize()
        x2, w2, b2 = fresh()
        with torch.no_grad():
            x2.copy_(embed[token] * (0.5 + k))
        assert all(torch.equal(p, q) for p, q in zip(got, step(x2, (w2, b2)))), k
