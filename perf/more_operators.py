"""The cases on which the gated projection, the 8-bit checkpoints and the
post-training losses are measured.

Four operators around DetLinear and token_logprobs: the gated projection
act(x Wg^T) * (x Wu^T) (serving, training, and training with its activations
kept in 8 bits), the 8-bit checkpoint itself (written and read back), the
clipped policy loss with a KL term and the preference loss over pairs, both
with their gradients.

run() computes them in their plain form, elementary torch operations in 32
bits rounded once at the end (in 64 where a difference or a border asks for
it), or through this package's entry points when `own` is set.  exact() gives
the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


# --------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a serving loop: both weights are read once, nothing else counts
        {"name": "gated one token", "op": "gated", "N": 1, "C": 4096, "F": 11008, "y": "bf16", "act": "silu"},
        # a decoding batch of a small model with an odd hidden width
        {"name": "gated decode batch", "op": "gated", "N": 48, "C": 2048, "F": 5461, "y": "bf16", "act": "gelu_tanh"},
        # the tokens of a prompt
        {"name": "gated prompt", "op": "gated", "N": 8192, "C": 4096, "F": 11008, "y": "bf16", "act": "silu"},
        # a small training step, every size odd, fp32 out
        {"name": "gated train odd", "op": "gated_train", "N": 1021, "C": 1537, "F": 4099, "y": "f32", "act": "gelu"},
        # a large training step
        {"name": "gated train large", "op": "gated_train", "N": 8192, "C": 4096, "F": 11008, "y": "bf16",
         "act": "silu"},
        # the same with x and both projections kept in 8 bits for the backward pass
        {"name": "gated train int8", "op": "gated_int8", "N": 8192, "C": 4096, "F": 11008, "y": "bf16",
         "act": "silu"},
        # a few fp32 rows whose last block is ragged
        {"name": "checkpoint small", "op": "pack", "N": 64, "C": 1001, "x": "f32", "y": "f32"},
        # the input of a wide layer over a batch of tokens
        {"name": "checkpoint large", "op": "pack", "N": 16384, "C": 8192, "x": "bf16", "y": "bf16"},
        # one prompt's group of sampled answers
        {"name": "policy small", "op": "policy", "B": 8, "T": 300, "kl": 0.0, "per_token": False,
         "reduction": "sequences"},
        # a large batch of ragged answers with a reference model and per-token advantages
        {"name": "policy large", "op": "policy", "B": 1024, "T": 8192, "kl": 0.05, "per_token": True,
         "reduction": "tokens"},
        # a small batch of pairs of answers
        {"name": "preference small", "op": "preference", "P": 16, "Tc": 128, "Tr": 150, "kind": "sigmoid",
         "smooth": 0.1},
        # a large one, answers padded to two lengths
        {"name": "preference large", "op": "preference", "P": 2048, "Tc": 4096, "Tr": 2049, "kind": "sigmoid",
         "smooth": 0.0},
    ]


def _log_size(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_train", "gated_int8", "pack", "policy", "preference"])
    if op.startswith("gated"):
        C, F = _log_size(rng, 64, 8192), _log_size(rng, 64, 11008)
        if rng.random() < 0.5:              # most models' widths are multiples of 64
            C, F = (C + 63) // 64 * 64, (F + 63) // 64 * 64
        N = _log_size(rng, 1, min(8192, 8192 * 4096 * 11008 // (C * F)))
        return {"op": op, "N": N, "C": C, "F": F, "y": rng.choice(["bf16", "f32"]),
                "act": rng.choice(["silu", "gelu", "gelu_tanh"])}
    if op == "pack":
        C = _log_size(rng, 8, 16384)
        return {"op": op, "N": _log_size(rng, 1, min(2 ** 17, 2 ** 27 // C)), "C": C,
                "x": rng.choice(["f32", "bf16"]), "y": rng.choice(["f32", "bf16"])}
    if op == "policy":
        T = _log_size(rng, 1, 16384)
        return {"op": op, "B": _log_size(rng, 1, min(2048, 2 ** 23 // T)), "T": T, "kl": rng.choice([0.0, 0.05]),
                "per_token": rng.random() < 0.5, "reduction": rng.choice(["tokens", "sequences", "none"])}
    Tc, Tr = _log_size(rng, 1, 8192), _log_size(rng, 1, 8192)
    kind = rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"])
    return {"op": op, "P": _log_size(rng, 1, min(2048, 2 ** 23 // max(Tc, Tr))), "Tc": Tc, "Tr": Tr, "kind": kind,
            "smooth": rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0}


# -------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _gated_inputs(c, seed):
    """A norm's output, weights of a layer's usual spread, and a gradient for each of its outputs."""
    g = _gen(seed)
    N, C, F = c["N"], c["C"], c["F"]
    bf16 = torch.bfloat16
    x = (_randn(g, N, C) * (1.0 + 0.2 * _randn(g, C))).to(bf16)
    wg, wu = ((_randn(g, F, C) / math.sqrt(C)).to(bf16) for _ in range(2))
    dh = None if c["op"] == "gated" else (_randn(g, N, F) / math.sqrt(N)).to(_DT[c["y"]])
    return x, wg, wu, dh


def _pack_inputs(c, seed):
    """Activations: a spread per channel, some channels far above the others, one row of zeros."""
    g = _gen(seed)
    x = _randn(g, c["N"], c["C"]) * torch.exp(0.5 * _randn(g, c["C"]))
    x = x * torch.where(torch.rand(c["C"], generator=g, device="cuda") < 0.01, 30.0, 1.0)
    x[c["N"] // 2] = 0.0
    return x.to(_DT[c["x"]])


def _answers(g, rows, T, empty):
    """Log probabilities of sampled tokens, valid up to each row's length; what lies behind is not finite."""
    length = torch.randint(max(1, T // 4), T + 1, (rows, 1), generator=g, device="cuda")
    if empty and rows > 4:
        length[rows // 2] = 0               # an answer whose mask leaves nothing
    mask = torch.arange(T, device="cuda") < length
    lp = -torch.abs(1.5 * _randn(g, rows, T))
    return lp.masked_fill_(~mask, float("nan")), mask


def _policy_inputs(c, seed):
    g = _gen(seed)
    lp, mask = _answers(g, c["B"], c["T"], True)
    old = lp + 0.2 * _randn(g, c["B"], c["T"])
    ref = lp + 0.3 * _randn(g, c["B"], c["T"]) if c["kl"] else None
    adv = _randn(g, c["B"], c["T"]) if c["per_token"] else _randn(g, c["B"])
    weight = torch.rand(c["B"], c["T"], generator=g, device="cuda") if c["reduction"] == "none" else None
    return lp, old, adv, mask, ref, weight


def _preference_inputs(c, seed):
    g = _gen(seed)
    sides = []
    for T in (c["Tc"], c["Tr"]):
        lp, mask = _answers(g, c["P"], T, True)
        sides.append((lp, lp + 0.3 * _randn(g, c["P"], T), mask))
    return sides, torch.rand(c["P"], generator=g, device="cuda") / c["P"]


def prepare(case, seed):
    c = dict(case)
    if c["op"].startswith("gated"):
        x, wg, wu, dh = _gated_inputs(c, seed)
        if dh is not None:
            x, wg, wu = (t.requires_grad_(True) for t in (x, wg, wu))
        return {"c": c, "x": x, "wg": wg, "wu": wu, "dh": dh}
    if c["op"] == "pack":
        return {"c": c, "x": _pack_inputs(c, seed)}
    if c["op"] == "policy":
        lp, old, adv, mask, ref, weight = _policy_inputs(c, seed)
        return {"c": c, "lp": lp.requires_grad_(True), "old": old, "adv": adv, "mask": mask, "ref": ref,
                "weight": weight}
    sides, grad = _preference_inputs(c, seed)
    return {"c": c, "sides": [(lp.requires_grad_(True), ref, mask) for lp, ref, mask in sides], "grad": grad}


CLIP_LOW, CLIP_HIGH, BETA = 0.2, 0.28, 0.1


# ---------------------------------------------------------- the plain forms

def _plain_act(kind, g):
    """(act(g), act'(g))"""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_int8(t):
    """t (fp32) as its 8-bit checkpoint stands for it: blocks of 32, codes of up to 127 and a power of two."""
    N, C = t.shape
    b = torch.nn.functional.pad(t, (0, -C % 32)).view(N, -1, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    # the least power that keeps the largest magnitude below 127.5 codes
    e = (((top.view(torch.int32) + 0x10000) >> 23) - 133).clamp(-126, 121)
    unit = ((e + 127) << 23).view(torch.float32)            # 2^e from its bits
    return (torch.round(b / unit).clamp(-127.0, 127.0) * unit).view(N, -1)[:, :C]


def _plain_gated(s):
    c = s["c"]
    x, wg, wu = (s[k].detach().float() for k in ("x", "wg", "wu"))
    g, u = x @ wg.t(), x @ wu.t()
    a, d = _plain_act(c["act"], g)
    out = {"h": (a * u).to(_DT[c["y"]])}
    if s["dh"] is None:
        return out
    dh = s["dh"].float()
    if c["op"] == "gated_int8":
        x, g, u = _plain_int8(x), _plain_int8(g), _plain_int8(u)
        a, d = _plain_act(c["act"], g)
    dg, du = dh * u * d, dh * a
    bf16 = torch.bfloat16
    out["dx"] = (dg @ wg + du @ wu).to(bf16)
    out["dwg"], out["dwu"] = (dg.t() @ x).to(bf16), (du.t() @ x).to(bf16)
    return out


def _plain_policy(s):
    c, mask = s["c"], s["mask"]
    lp, old = (torch.where(mask, s[k].detach(), 0.0).double() for k in ("lp", "old"))
    adv = s["adv"] if c["per_token"] else s["adv"][:, None]
    adv = torch.where(mask, adv, 0.0)
    d = lp - old                            # 64 bits: a token next to a bound of the clipping
    clipped = ((adv > 0.0) & (d > math.log1p(CLIP_HIGH))) | ((adv < 0.0) & (d < math.log1p(-CLIP_LOW)))
    r = torch.exp(d).float()
    bound = torch.where(adv > 0.0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    loss = -torch.where(clipped, bound, r) * adv
    slope = torch.where(clipped, 0.0, -r * adv)
    kl = torch.zeros_like(loss)
    if c["kl"]:
        q = torch.where(mask, s["ref"], 0.0).double() - lp
        kl = (torch.exp(q) - 1.0 - q).float()              # 64 bits: differences near 0
        loss = loss + c["kl"] * kl
        slope = slope + c["kl"] * (1.0 - torch.exp(q)).float()
    loss, kl, clipped, slope = (torch.where(mask, t, 0.0) for t in (loss, kl, clipped.float(), slope))
    if c["reduction"] == "none":
        return {"loss": loss, "kl": kl, "clipped": clipped, "dlp": slope * s["weight"]}
    n = mask.sum(dim=1)
    if c["reduction"] == "tokens":
        w = (1.0 / n.sum().clamp(min=1).double()).expand(c["B"], 1)
    else:
        w = (1.0 / (n.clamp(min=1) * (n > 0).sum().clamp(min=1)).double())[:, None]
    out = {k: (t.double() * w).sum().float() for k, t in (("loss", loss), ("kl", kl), ("clipped", clipped))}
    out["dlp"] = slope * w.float()
    return out


def _plain_preference(s):
    c = s["c"]
    sums = []
    for lp, ref, mask in s["sides"]:
        d = torch.where(mask, lp.detach().double() - ref.double(), 0.0)
        sums.append(d.sum(dim=1))           # 64 bits: long sums whose difference counts
    margin = sums[0] - sums[1]
    z = (BETA * margin).float()
    if c["kind"] == "sigmoid":
        e = torch.exp(-torch.abs(z))
        soft = torch.log1p(e)               # -ln sigmoid(|z|)
        neg = torch.where(z > 0.0, soft, soft - z)
        loss = (1.0 - c["smooth"]) * neg + c["smooth"] * (neg + z)
        wrong = torch.where(z > 0.0, e, 1.0) / (1.0 + e)   # sigmoid(-z)
        slope = BETA * (c["smooth"] - wrong)
    elif c["kind"] == "hinge":
        loss = torch.clamp(1.0 - z, min=0.0)
        slope = torch.where(z < 1.0, -BETA, 0.0)
    else:
        off = (margin - 1.0 / (2.0 * BETA)).float()
        loss, slope = off * off, 2.0 * off
    slope = (slope * s["grad"])[:, None]
    return {"loss": loss, "chosen": (BETA * sums[0]).float(), "rejected": (BETA * sums[1]).float(),
            "dchosen": torch.where(s["sides"][0][2], slope, 0.0), "drejected": torch.where(s["sides"][1][2], -slope, 0.0)}


# -------------------------------------------------------- the entry points

def _own_gated(s):
    import bitwise_deterministic_exact_amd as det
    c = s["c"]
    h = det.gated_linear(s["x"], s["wg"], s["wu"], activation=c["act"], out_dtype=_DT[c["y"]],
                         checkpoint="int8" if c["op"] == "gated_int8" else None)
    if s["dh"] is None:
        return {"h": h}
    dx, dwg, dwu = torch.autograd.grad(h, (s["x"], s["wg"], s["wu"]), s["dh"])
    return {"h": h.detach(), "dx": dx, "dwg": dwg, "dwu": dwu}


def _own_pack(s):
    import bitwise_deterministic_exact_amd as det
    return {"values": det.unpack_int8(det.pack_int8(s["x"]), dtype=_DT[s["c"]["y"]])}


def _own_policy(s):
    import bitwise_deterministic_exact_amd as det
    c = s["c"]
    r = det.policy_loss(s["lp"], s["old"], s["adv"], s["mask"], ref_logprob=s["ref"], clip_low=CLIP_LOW,
                        clip_high=CLIP_HIGH, kl_weight=c["kl"], reduction=c["reduction"])
    dlp, = torch.autograd.grad(r.loss, s["lp"], s["weight"])
    return {"loss": r.loss.detach(), "kl": r.kl, "clipped": r.clipped, "dlp": dlp}


def _own_preference(s):
    import bitwise_deterministic_exact_amd as det
    c, ((lc, rc, mc), (lr, rr, mr)) = s["c"], s["sides"]
    r = det.preference_loss(lc, lr, rc, rr, chosen_mask=mc, rejected_mask=mr, beta=BETA, kind=c["kind"],
                            label_smoothing=c["smooth"])
    dc, dr = torch.autograd.grad(r.loss, (lc, lr), s["grad"])
    return {"loss": r.loss.detach(), "chosen": r.chosen_reward, "rejected": r.rejected_reward, "dchosen": dc,
            "drejected": dr}


def run(state):
    op = state["c"]["op"]
    if op.startswith("gated"):
        return (_own_gated if own else _plain_gated)(state)
    if op == "pack":
        if own:
            return _own_pack(state)
        return {"values": _plain_int8(state["x"].float()).to(_DT[state["c"]["y"]])}
    if op == "policy":
        return (_own_policy if own else _plain_policy)(state)
    return (_own_preference if own else _plain_preference)(state)


# ----------------------------------------------------- the work, and 64 bits

def work(case):
    c = case
    if c["op"].startswith("gated"):
        N, C, F, sy = c["N"], c["C"], c["F"], _SIZE[c["y"]]
        fwd = {"bytes": 2 * (N * C + 2 * F * C) + N * F * sy, "flops": 4 * N * C * F}
        if c["op"] == "gated":
            return fwd
        # dh read, dx and both weights' gradients written
        return {"bytes": fwd["bytes"] + N * F * sy + 2 * (N * C + 2 * F * C), "flops": 12 * N * C * F}
    if c["op"] == "pack":
        n = c["N"] * c["C"]
        return {"bytes": n * (_SIZE[c["x"]] + _SIZE[c["y"]]) + 2 * c["N"] * (c["C"] + (c["C"] + 31) // 32),
                "flops": 4 * n}
    if c["op"] == "policy":
        n = c["B"] * c["T"]
        arrays = 3 + (c["kl"] > 0.0) + c["per_token"] + (4 if c["reduction"] == "none" else 0) - (
            c["reduction"] == "none")
        return {"bytes": n * (4 * arrays + 1), "flops": 20 * n}
    n = c["P"] * (c["Tc"] + c["Tr"])
    return {"bytes": n * 13, "flops": 4 * n}


def _exact_act(kind, g):
    F = torch.nn.functional
    return F.silu(g) if kind == "silu" else F.gelu(g, approximate="none" if kind == "gelu" else "tanh")


def _exact_int8(t):
    N, C = t.shape
    pad = -C % 32
    b = torch.cat([t, t.new_zeros(N, pad)], dim=1).unflatten(1, (-1, 32))
    top = b.abs().max(dim=2, keepdim=True).values
    m, k = torch.frexp(top)                 # top = m 2^k, 1/2 <= m < 1
    e = k.double() - 7.0 + (m * 128.0 >= 127.5)
    e = torch.where(top == 0.0, -126.0, e).clamp(-126.0, 121.0)
    unit = ((e.long() + 1023) << 52).view(torch.float64)    # pow(2, e) is off by a unit: ties would break
    return ((b / unit).round().clamp(-127.0, 127.0) * unit).flatten(1)[:, :C]


def _exact_gated(c, seed):
    x, wg, wu, dh = _gated_inputs(c, seed)
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    out = {"h": _exact_act(c["act"], g) * u}
    if dh is None:
        return out
    if c["op"] == "gated_int8":
        x, g, u = _exact_int8(x), _exact_int8(g), _exact_int8(u)
    g, u = g.requires_grad_(True), u.requires_grad_(True)
    dg, du = torch.autograd.grad(_exact_act(c["act"], g) * u, (g, u), dh.double())
    out["dx"] = dg @ wg + du @ wu
    out["dwg"], out["dwu"] = dg.t() @ x, du.t() @ x
    return out


def _exact_policy(c, seed):
    lp, old, adv, mask, ref, weight = _policy_inputs(c, seed)
    lp = lp.double().masked_fill(~mask, 0.0).requires_grad_(True)
    old = old.double().masked_fill(~mask, 0.0)
    adv = (adv if c["per_token"] else adv[:, None].expand_as(lp)).double()
    r = torch.exp(lp - old)
    a, b = r * adv, r.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH) * adv
    loss, clipped = -torch.where(a <= b, a, b), (a > b).double()
    kl = torch.zeros_like(loss)
    if c["kl"]:
        q = ref.double().masked_fill(~mask, 0.0) - lp
        kl = torch.expm1(q) - q
        loss = loss + c["kl"] * kl
    loss, kl, clipped = (t.masked_fill(~mask, 0.0) for t in (loss, kl, clipped))
    if c["reduction"] == "tokens":
        loss, kl, clipped = (t.sum() / max(1, int(mask.sum())) for t in (loss, kl, clipped))
    elif c["reduction"] == "sequences":
        n = mask.sum(dim=1)
        some = max(1, int((n > 0).sum()))
        loss, kl, clipped = ((t.sum(dim=1) / n.clamp(min=1)).sum() / some for t in (loss, kl, clipped))
    dlp, = torch.autograd.grad(loss, lp, None if weight is None else weight.double())
    return {"loss": loss.detach(), "kl": kl.detach(), "clipped": clipped, "dlp": dlp}


def _exact_preference(c, seed):
    (chosen, rejected), grad = _preference_inputs(c, seed)
    leaves, sums = [], []
    for lp, ref, mask in (chosen, rejected):
        leaves.append(lp.double().masked_fill(~mask, 0.0).requires_grad_(True))
        sums.append((leaves[-1] - ref.double().masked_fill(~mask, 0.0)).masked_fill(~mask, 0.0).sum(dim=1))
    margin = sums[0] - sums[1]
    if c["kind"] == "sigmoid":
        logsig = torch.nn.functional.logsigmoid
        loss = -(1.0 - c["smooth"]) * logsig(BETA * margin) - c["smooth"] * logsig(-BETA * margin)
    elif c["kind"] == "hinge":
        loss = torch.relu(1.0 - BETA * margin)
    else:
        loss = (margin - 1.0 / (2.0 * BETA)) ** 2
    dc, dr = torch.autograd.grad(loss, leaves, grad.double())
    return {"loss": loss.detach(), "chosen": BETA * sums[0].detach(), "rejected": BETA * sums[1].detach(),
            "dchosen": dc, "drejected": dr}


def exact(case, seed):
    c = dict(case)
    if c["op"].startswith("gated"):
        return _exact_gated(c, seed)
    if c["op"] == "pack":
        return {"values": _exact_int8(_pack_inputs(c, seed).double())}
    return (_exact_policy if c["op"] == "policy" else _exact_preference)(c, seed)
