"""The cases on which the language-model-head operators are measured.

Three operators that a training or scoring step calls one after another around
a DetLinear head: layer norm (forward, and with its backward pass), the log
probabilities of given tokens with entropy and top alternatives (for scoring,
and with their backward pass), and distillation from a teacher's top logits
(forward and backward).

run() computes them in their plain form, elementary torch operations in 32
bits rounded once at the end, or through this package's entry points when
`own` is set.  exact() gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NEG_INF = float("-inf")


# --------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving loop through the norm: all latency
        {"name": "norm one token", "op": "norm", "N": 1, "C": 4096, "x": "bf16", "y": "bf16", "w": "bf16"},
        # 8192 tokens of a DetLinear's fp32 output on the way into the next bf16 DetLinear
        {"name": "norm f32 to bf16", "op": "norm", "N": 8192, "C": 4096, "x": "f32", "y": "bf16", "w": "bf16"},
        # a small fp32 training step with an odd width and row count
        {"name": "norm train odd", "op": "norm_train", "N": 1021, "C": 1537, "x": "f32", "y": "f32", "w": "f32"},
        # a large bf16 training step
        {"name": "norm train large", "op": "norm_train", "N": 16384, "C": 8192, "x": "bf16", "y": "bf16", "w": "bf16"},
        # one token of a serving loop: its log probability, the entropy and 20 alternatives
        {"name": "score one token", "op": "score", "N": 1, "V": 131072, "x": "f32", "top": 20, "scale": 1.0,
         "masked": False},
        # a decoding batch over an odd vocabulary with banned tokens, at a temperature of 0.8
        {"name": "score batch", "op": "score", "N": 64, "V": 50257, "x": "bf16", "top": 5, "scale": 1.25,
         "masked": True},
        # the tokens of collected rollouts scored again before a policy update
        {"name": "score rollouts", "op": "score", "N": 4096, "V": 131072, "x": "bf16", "top": 0, "scale": 1.0,
         "masked": False},
        # a small classification-sized training step
        {"name": "score train small", "op": "score_train", "N": 512, "V": 1000, "x": "f32", "top": 0, "scale": 1.0,
         "masked": False},
        # a policy-gradient step with an entropy bonus on a DetLinear head's fp32 logits, odd vocabulary
        {"name": "score train", "op": "score_train", "N": 2048, "V": 100003, "x": "f32", "top": 0, "scale": 1.0,
         "masked": True},
        # a small student on a small vocabulary
        {"name": "distill small", "op": "distill", "N": 128, "V": 4096, "x": "bf16", "K": 8, "temperature": 1.0},
        # fp32 logits, odd vocabulary and entry count, a softened teacher
        {"name": "distill odd", "op": "distill", "N": 1021, "V": 50257, "x": "f32", "K": 33, "temperature": 2.0},
        # a large bf16 step against 64 entries per token
        {"name": "distill large", "op": "distill", "N": 4096, "V": 131072, "x": "bf16", "K": 64, "temperature": 1.0},
    ]


def _log_size(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "score", "score_train", "distill"])
    if op.startswith("norm"):
        C = _log_size(rng, 16, 16384)
        N = _log_size(rng, 1, min(16384, 2 ** 27 // C))
        x = rng.choice(["f32", "bf16"])
        y = rng.choice(["f32", "bf16"])
        return {"op": op, "N": N, "C": C, "x": x, "y": y, "w": rng.choice(["f32", "bf16"])}
    V = _log_size(rng, 64, 200000)
    N = _log_size(rng, 1, min(4096, 2 ** 28 // V))
    x = rng.choice(["f32", "bf16"])
    if op == "distill":
        return {"op": op, "N": N, "V": V, "x": x, "K": _log_size(rng, 1, min(V, 128)),
                "temperature": rng.choice([0.5, 1.0, 2.0, 4.0])}
    top = rng.choice([0, 1, 5, 20, 50]) if op == "score" else 0
    return {"op": op, "N": N, "V": V, "x": x, "top": top, "scale": rng.choice([1.0, 1.25, 0.5]),
            "masked": rng.random() < 0.5}


# -------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _norm_inputs(c, seed):
    """Hidden states with a per-channel offset, weights near one, biases near zero."""
    g = _gen(seed)
    N, C = c["N"], c["C"]
    x = (_randn(g, N, C) * 1.5 + 0.5 * _randn(g, C)).to(_DT[c["x"]])
    w = (1.0 + 0.1 * _randn(g, C)).to(_DT[c["w"]])
    b = (0.1 * _randn(g, C)).to(_DT[c["w"]])
    dy = (_randn(g, N, C) / math.sqrt(N)).to(_DT[c["y"]]) if c["op"] == "norm_train" else None
    return x, w, b, dy


def _logits(c, g, targets=None):
    """Head outputs: normal noise, with the given tokens lifted in most rows."""
    N, V = c["N"], c["V"]
    z = _randn(g, N, V).mul_(2.5)
    if targets is not None:
        z.scatter_add_(1, targets.reshape(N, -1), 4.0 + 2.0 * _randn(g, N, targets.numel() // N))
    return z


def _score_inputs(c, seed):
    g = _gen(seed)
    N, V = c["N"], c["V"]
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    z = _logits(c, g, t)
    if c["masked"]:
        # a ban list shared by the batch, and one row that it leaves nothing
        z.masked_fill_(torch.rand(V, generator=g, device="cuda") < 0.05, NEG_INF)
        if N > 8:
            z[N // 2] = NEG_INF
    glp = _randn(g, N) / N
    gent = torch.full((N,), -0.01 / N, device="cuda") * (1.0 + torch.rand(N, generator=g, device="cuda"))
    return z.to(_DT[c["x"]]), t, glp, gent


def _distill_inputs(c, seed):
    """A teacher's K highest logits per token, in descending order, with their token numbers."""
    g = _gen(seed)
    N, V, K = c["N"], c["V"], c["K"]
    first = torch.randint(0, V, (N, 1), generator=g, device="cuda")
    step = 2 * torch.randint(0, max(1, V // (2 * K)), (N, 1), generator=g, device="cuda") + 1
    idx = (first + step * torch.arange(K, device="cuda")) % V
    teacher = (2.0 * _randn(g, N, K) + 6.0).sort(dim=1, descending=True).values
    z = _randn(g, N, V).mul_(2.0)
    z.scatter_add_(1, idx, 0.5 * teacher)
    grad = torch.rand(N, generator=g, device="cuda") / N
    return z.to(_DT[c["x"]]), teacher, idx, grad


def prepare(case, seed):
    c = dict(case)
    if c["op"].startswith("norm"):
        x, w, b, dy = _norm_inputs(c, seed)
        if dy is not None:
            x, w, b = (t.requires_grad_(True) for t in (x, w, b))
        return {"c": c, "x": x, "w": w, "b": b, "dy": dy}
    if c["op"] == "distill":
        z, teacher, idx, grad = _distill_inputs(c, seed)
        return {"c": c, "z": z.requires_grad_(True), "teacher": teacher, "idx": idx, "grad": grad}
    z, t, glp, gent = _score_inputs(c, seed)
    return {"c": c, "z": z.requires_grad_(c["op"] == "score_train"), "t": t, "glp": glp, "gent": gent}


# ---------------------------------------------------------- the plain forms

EPS = 1e-5


def _plain_norm(s):
    c = s["c"]
    x, w, b = (s[k].detach().float() for k in ("x", "w", "b"))
    d = x - x.mean(dim=1, keepdim=True)
    r = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    h = d * r
    y = (h * w + b).to(_DT[c["y"]])
    if s["dy"] is None:
        return {"y": y}
    dy = s["dy"].float()
    g = dy * w
    dx = r * (g - g.mean(dim=1, keepdim=True) - h * (g * h).mean(dim=1, keepdim=True))
    return {"y": y, "dx": dx.to(_DT[c["x"]]), "dw": (dy * h).sum(dim=0).to(_DT[c["w"]]),
            "db": dy.sum(dim=0).to(_DT[c["w"]])}


def _plain_top(raw, k):
    """The k largest of each row, ties to the lowest index: the order of the
    fp32 bit patterns and the index packed into one integer key."""
    b = (raw + 0.0).view(torch.int32).to(torch.int64)
    order = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
    key = order * (1 << 31) + (raw.shape[1] - 1 - torch.arange(raw.shape[1], device=raw.device))
    top = torch.topk(key, k, dim=1).values
    return raw.shape[1] - 1 - torch.remainder(top, 1 << 31)


def _plain_softmax(raw, scale):
    """(log-probabilities, probabilities) in 32 bits; a row of nothing but
    -inf has the log probability -inf and the probability 0 everywhere."""
    m = raw.amax(dim=1, keepdim=True)
    d = (raw - torch.where(m == NEG_INF, 0.0, m)) * scale
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    total = torch.where(total == 0.0, 1.0, total)
    return d - torch.log(total), e / total


def _plain_score(s):
    c = s["c"]
    raw, t = s["z"].detach().float(), s["t"][:, None]
    lp, p = _plain_softmax(raw, c["scale"])
    plp = p * torch.where(p > 0.0, lp, 0.0)
    ent = -plp.sum(dim=1)
    out = {"logprob": lp.gather(1, t)[:, 0], "entropy": ent}
    if c["top"]:
        out["top_index"] = _plain_top(raw, c["top"])
        out["top_logprob"] = lp.gather(1, out["top_index"])
    if c["op"] == "score_train":
        empty = raw.amax(dim=1, keepdim=True) == NEG_INF
        glp, gent = s["glp"][:, None], s["gent"][:, None]
        dz = -p * (glp + gent * ent[:, None]) - gent * plp
        dz.scatter_add_(1, t, glp)
        out["dz"] = (torch.where(empty, 0.0, dz) * c["scale"]).to(s["z"].dtype)
    return out


def _plain_distill(s):
    c = s["c"]
    T = c["temperature"]
    lp, p = _plain_softmax(s["z"].detach().float(), 1.0 / T)
    lq, q = _plain_softmax(s["teacher"].float(), 1.0 / T)
    loss = T * T * (q * (lq - lp.gather(1, s["idx"]))).sum(dim=1)
    p.scatter_add_(1, s["idx"], -q)
    return {"loss": loss, "dz": (p * (T * s["grad"][:, None])).to(s["z"].dtype)}


# -------------------------------------------------------- the entry points

def _own_norm(s):
    import bitwise_deterministic_exact_amd as det
    y = det.layer_norm(s["x"], s["w"], s["b"], eps=EPS, out_dtype=_DT[s["c"]["y"]])
    if s["dy"] is None:
        return {"y": y}
    dx, dw, db = torch.autograd.grad(y, (s["x"], s["w"], s["b"]), s["dy"])
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}


def _own_score(s):
    import bitwise_deterministic_exact_amd as det
    c = s["c"]
    r = det.token_logprobs(s["z"], s["t"], scale=c["scale"], top=c["top"])
    out = {"logprob": r.logprob.detach(), "entropy": r.entropy.detach()}
    if c["top"]:
        out["top_index"], out["top_logprob"] = r.top_index, r.top_logprob.detach()
    if c["op"] == "score_train":
        out["dz"], = torch.autograd.grad((r.logprob, r.entropy), s["z"], (s["glp"], s["gent"]))
    return out


def _own_distill(s):
    import bitwise_deterministic_exact_amd as det
    loss = det.distill_loss(s["z"], s["teacher"], s["idx"], temperature=s["c"]["temperature"])
    dz, = torch.autograd.grad(loss, s["z"], s["grad"])
    return {"loss": loss.detach(), "dz": dz}


def run(state):
    op = state["c"]["op"]
    if own:
        return (_own_norm if op.startswith("norm") else _own_distill if op == "distill" else _own_score)(state)
    return (_plain_norm if op.startswith("norm") else _plain_distill if op == "distill" else _plain_score)(state)


# ----------------------------------------------------- the work, and 64 bits

_SIZE = {"f32": 4, "bf16": 2}


def work(case):
    c = case
    if c["op"].startswith("norm"):
        N, C, sx, sy, sw = c["N"], c["C"], _SIZE[c["x"]], _SIZE[c["y"]], _SIZE[c["w"]]
        n = N * C
        fwd = {"bytes": n * (sx + sy) + 2 * C * sw, "flops": 8 * n}
        if c["op"] == "norm":
            return fwd
        # x and dy read once, y and dx written once, the weights' gradients written
        return {"bytes": n * (2 * sx + 2 * sy) + 4 * C * sw, "flops": 22 * n}
    n, sx = c["N"] * c["V"], _SIZE[c["x"]]
    if c["op"] == "distill":
        return {"bytes": 2 * n * sx + c["N"] * (c["K"] * 12 + 8), "flops": 8 * n}
    if c["op"] == "score":
        return {"bytes": n * sx + c["N"] * (16 + c["top"] * 12), "flops": 6 * n}
    return {"bytes": 2 * n * sx + c["N"] * 24, "flops": 13 * n}


def _exact_norm(c, seed):
    x, w, b, dy = _norm_inputs(c, seed)
    x, w, b = (t.double().requires_grad_(dy is not None) for t in (x, w, b))
    var, mean = torch.var_mean(x, dim=1, keepdim=True, unbiased=False)
    y = (x - mean) * torch.rsqrt(var + EPS) * w + b
    if dy is None:
        return {"y": y}
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy.double())
    return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}


def _exact_score(c, seed):
    z0, t, glp, gent = _score_inputs(c, seed)
    masked = torch.isneginf(z0)
    empty = masked.all(dim=1)
    z = z0.double()
    z[empty] = 0.0
    z.requires_grad_(c["op"] == "score_train")
    lp = torch.log_softmax(z * c["scale"], dim=1)
    ent = -(lp.exp() * lp.masked_fill(masked, 0.0)).sum(dim=1)
    logprob = lp.gather(1, t[:, None])[:, 0]
    out = {"logprob": logprob.detach().masked_fill(empty, NEG_INF), "entropy": ent.detach().masked_fill(empty, 0.0)}
    if c["top"]:
        out["top_index"] = torch.sort(z0.double(), dim=1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_logprob"] = lp.detach().gather(1, out["top_index"]).masked_fill(empty[:, None], NEG_INF)
    if c["op"] == "score_train":
        dz, = torch.autograd.grad((logprob, ent), z, (glp.double(), gent.double()))
        out["dz"] = dz.masked_fill(empty[:, None], 0.0)
    return out


def _exact_distill(c, seed):
    z, teacher, idx, grad = _distill_inputs(c, seed)
    T = c["temperature"]
    z = z.double().requires_grad_(True)
    lp = torch.log_softmax(z / T, dim=1).gather(1, idx)
    lq = torch.log_softmax(teacher.double() / T, dim=1)
    loss = T * T * (lq.exp() * (lq - lp)).sum(dim=1)
    dz, = torch.autograd.grad(loss, z, grad.double())
    return {"loss": loss.detach(), "dz": dz}


def exact(case, seed):
    c = dict(case)
    if c["op"].startswith("norm"):
        return _exact_norm(c, seed)
    return _exact_distill(c, seed) if c["op"] == "distill" else _exact_score(c, seed)
