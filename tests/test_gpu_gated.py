"""The gated projection on the GPU: products bit for bit on integers, h and the
gradients against 64 bits, batch independence, layouts, checkpoints in 8 bits,
differences, streams and graph replays."""
import math

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
# a rounding is off by at most half a step of the value
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
# fp32 sums of n products: at most this relative to the sum of their magnitudes,
# one rounding (of either kind, so a whole step) per addition
def sum_bound(n):
    return (n + 2) * 2.0 ** -23


ACTS = ("silu", "gelu", "gelu_tanh")
# few tokens (16, 32 and 64 at a time), tiles of 128 (ragged both ways, one and many steps of k, odd widths),
# tiles of 256 (ragged both ways)
SIZES = [(1, 64, 16), (1, 31, 1), (3, 1, 5), (16, 32, 33), (17, 100, 64), (33, 257, 130), (64, 192, 48), (48, 2048, 96),
         (65, 64, 64), (130, 128, 100), (129, 100, 257), (300, 512, 31), (200, 65, 200), (4100, 64, 2100),
         (2100, 192, 4099)]


def integers(g, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).to(BF16)


def operands(seed, N, C, F, normal=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if not normal:
        return integers(g, N, C), integers(g, F, C), integers(g, F, C)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    return r(N, C).to(BF16), (r(F, C) / math.sqrt(C)).to(BF16), (r(F, C) / math.sqrt(C)).to(BF16)


def act64(kind, g):
    if kind == "silu":
        return torch.nn.functional.silu(g)
    return torch.nn.functional.gelu(g, approximate="none" if kind == "gelu" else "tanh")


def slope64(kind, g):
    g = g.detach().requires_grad_(True)
    return torch.autograd.grad(act64(kind, g).sum(), g)[0]


def two(e):
    """2^e from its bits (pow is off by a unit of 64 bits)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def value(t):
    """What a kept projection stands for, in 64 bits."""
    if isinstance(t, det.PackedInt8):
        return det.unpack_int8(t).double()
    return t.values.double() * two(t.exponents).repeat_interleave(32, -1)[..., :t.values.shape[-1]]


def half64(v):
    """v (64 bits) as fp16 elements of blocks of 32: (values, exponents)."""
    N, F = v.shape
    b = torch.nn.functional.pad(v, (0, -F % 32)).reshape(N, -1, 32)
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    e = (torch.frexp(top)[1].long() - 15).clamp(min=-126)
    e = torch.where(top == 0, -126, e)
    h = (b * two(-e)[..., None]).to(torch.float16)     # a sum of few bits: rounded once
    return h.reshape(N, -1)[:, :F], e.to(torch.int8)


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{((got.double() - want).abs() / bound.clamp(min=1e-300)).max().item():.3g} of the bound")


@pytest.mark.parametrize("N,C,F", SIZES)
def test_products_are_exact_on_integers(N, C, F):
    # every partial sum is an integer below 2^24: g and u have to be exact
    announce(f"gated integers {N} {C} {F}")
    x, wg, wu = operands(1, N, C, F, normal=False)
    _, s = det.gated_linear_forward(x, wg, wu)
    for got, w in ((s.gate, wg), (s.up, wu)):
        values, exps = half64(x.double() @ w.double().t())
        assert torch.equal(got.values, values) and torch.equal(got.exponents, exps)
    # the same products where nothing is kept (few tokens take another kernel): act(g) ~ g from 32 on is g
    one = torch.zeros(F, C, device=DEV, dtype=BF16)
    one[:, 0] = 64.0
    x[:, 0] = 1.0
    h = det.gated_linear(x, one, wu, out_dtype=F32)
    assert torch.equal(h, 64.0 * (x.double() @ wu.double().t()).to(F32))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("N,C,F", SIZES)
def test_forward_against_64_bits(N, C, F, act, out):
    announce(f"gated forward {N} {C} {F} {act} {out}")
    x, wg, wu = operands(2, N, C, F)
    X, G, W = x.double(), wg.double(), wu.double()
    g, u = X @ G.t(), X @ W.t()
    eg, eu = (sum_bound(C) * (X.abs() @ w.abs().t()) for w in (G, W))
    a = act64(act, g)
    # |act'| <= 1.13; the activation and the product round a few times in 32 bits (8 half steps),
    # in the exponent too (another |g| of them)
    ea = 1.2 * eg + (8 + g.abs()) * U[F32] * a.abs() + 1e-37
    bound = ea * (u.abs() + eu) + a.abs() * eu + U[out] * (a * u).abs() * 1.01 + 1e-37
    h = det.gated_linear(x, wg, wu, activation=act, out_dtype=out)
    assert h.dtype == out
    within(h, a * u, bound, "h")
    kept, _ = det.gated_linear_forward(x, wg, wu, activation=act, out_dtype=out)
    assert torch.equal(h, kept)


def reference_grads(act, dh, x, wg, wu, g, u):
    """(value, bound) of dx, dw_gate, dw_up in 64 bits from the g and u that the gradient reads."""
    D, X, G, W = dh.double(), x.double(), wg.double(), wu.double()
    a, s = act64(act, g), slope64(act, g)
    dg, du = D * u * s, D * a
    # formed in 32 bits (8 half steps; the slope's parts may cancel: 8 of their sizes, |g| in the exponent), rounded to bf16
    eg = U[BF16] * dg.abs() * 1.01 + (8 + g.abs()) * U[F32] * (D * u).abs() * (1 + g.abs())
    eu = U[BF16] * du.abs() * 1.01 + (8 + g.abs()) * U[F32] * (D * g).abs()
    ag, au = dg.abs() + eg, du.abs() + eu
    out = []
    N, F = g.shape
    dx = dg @ G + du @ W
    out.append((dx, eg @ G.abs() + eu @ W.abs() + sum_bound(2 * F + 64) * (ag @ G.abs() + au @ W.abs()) + U[BF16] * dx.abs()))
    for d, e, m in ((dg, eg, ag), (du, eu, au)):
        w = d.t() @ X
        out.append((w, e.t() @ X.abs() + sum_bound(N + 64) * (m.t() @ X.abs()) + U[BF16] * w.abs()))
    return out


@pytest.mark.parametrize("act,dtype", [("silu", BF16), ("gelu", F32), ("gelu_tanh", BF16)])
@pytest.mark.parametrize("N,C,F", SIZES)
def test_gradients_against_64_bits(N, C, F, act, dtype):
    announce(f"gated gradients {N} {C} {F} {act} {dtype}")
    x, wg, wu = operands(3, N, C, F)
    dh = torch.randn(N, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)).to(dtype)
    h, s = det.gated_linear_forward(x, wg, wu, activation=act, out_dtype=dtype)
    got = det.gated_linear_backward(dh, x, wg, wu, s, activation=act)
    want = reference_grads(act, dh, x, wg, wu, value(s.gate), value(s.up))
    for name, t, (v, b) in zip(("dx", "dw_gate", "dw_up"), got, want):
        assert t.dtype == BF16
        within(t, v, b + 1e-37, name)
    # each alone, and through autograd: the same bits
    assert torch.equal(det.gated_linear_backward(dh, x, wg, wu, s, activation=act, need_dw=False)[0], got[0])
    only = det.gated_linear_backward(dh, x, wg, wu, s, activation=act, need_dx=False)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu)]
    again = det.gated_linear(*leaves, activation=act, out_dtype=dtype)
    assert torch.equal(again.detach(), h)
    for a, b in zip(torch.autograd.grad(again, leaves, dh), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N,C,F", [(1100, 130, 2500), (200, 1000, 2500), (2000, 512, 2816)])
def test_many_tiles_of_few_stages(N, C, F):
    test_products_are_exact_on_integers(N, C, F)
    test_gradients_against_64_bits(N, C, F, "silu", BF16)


@pytest.mark.parametrize("N,C,F", [(1, 31, 1), (17, 100, 64), (130, 128, 100), (300, 96, 33), (4100, 64, 2100)])
def test_int8_checkpoint(N, C, F):
    announce(f"gated int8 {N} {C} {F}")
    # integers: g and u are exact, and so are their codes
    x, wg, wu = operands(5, N, C, F, normal=False)
    _, s = det.gated_linear_forward(x, wg, wu, checkpoint="int8")
    for packed, w in ((s.gate, wg), (s.up, wu)):
        want = det.pack_int8((x.double() @ w.double().t()).to(F32))
        assert torch.equal(packed.codes, want.codes) and torch.equal(packed.exponents, want.exponents)
    x, wg, wu = operands(6, N, C, F)
    dh = torch.randn(N, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(7)).to(BF16)
    h, s = det.gated_linear_forward(x, wg, wu, checkpoint="int8")
    assert torch.equal(h, det.gated_linear_forward(x, wg, wu)[0])
    px = det.pack_int8(x)
    got = det.gated_linear_backward(dh, px, wg, wu, s)
    values = [det.unpack_int8(t).double() for t in (px, s.gate, s.up)]
    for name, t, (v, b) in zip(("dx", "dw_gate", "dw_up"), got,
                               reference_grads("silu", dh, values[0], wg, wu, values[1], values[2])):
        within(t, v, b + 1e-37, name)
    # what autograd does: the same, and the saved tensors are the 8-bit ones
    leaves = [t.clone().requires_grad_(True) for t in (x, wg, wu)]
    sizes = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append((t.dtype, t.numel())), t)[1], lambda t: t):
        again = det.gated_linear(*leaves, checkpoint="int8")
    kept = sum(n for d, n in sizes if d == torch.int8)
    assert kept == N * (C + 2 * F) + N * ((C + 31) // 32 + 2 * ((F + 31) // 32))
    assert sum(n for d, n in sizes if d != torch.int8) == 2 * F * C        # the weights
    for a, b in zip(torch.autograd.grad(again, leaves, dh), got):
        assert torch.equal(a, b)
    # a packed x with projections in 16 bits, too
    _, sb = det.gated_linear_forward(x, wg, wu)
    mixed = det.gated_linear_backward(dh, px, wg, wu, sb)
    plain = det.gated_linear_backward(dh, x, wg, wu, sb)
    assert torch.equal(mixed[0], plain[0])
    full = det.gated_linear_backward(dh, det.unpack_int8(px, BF16), wg, wu, sb)
    assert torch.equal(mixed[1], full[1]) and torch.equal(mixed[2], full[2])


@pytest.mark.parametrize("C,F", [(64, 2100), (100, 70), (192, 4099)])
def test_a_token_is_the_same_in_any_batch(C, F):
    # few tokens, tiles of 128 and of 256 rows: one chain of sums
    x, wg, wu = operands(8, 4100, C, F)
    dh = torch.randn(4100, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(9))
    h, s = det.gated_linear_forward(x, wg, wu, out_dtype=F32)
    dx = det.gated_linear_backward(dh, x, wg, wu, s, need_dw=False)[0]
    for a, b in ((0, 1), (4099, 4100), (5, 21), (100, 164), (64, 193), (1000, 1700)):
        part, t = det.gated_linear_forward(x[a:b], wg, wu, out_dtype=F32)
        assert torch.equal(part, h[a:b])
        assert torch.equal(det.gated_linear(x[a:b], wg, wu, out_dtype=F32), h[a:b])
        assert torch.equal(det.gated_linear_backward(dh[a:b], x[a:b], wg, wu, t, need_dw=False)[0], dx[a:b])


@pytest.mark.parametrize("N,C,F", [(1100, 1024, 700), (1021, 1537, 900), (520, 4100, 640), (90, 200, 129), (3000, 70, 65)])
def test_dx_of_a_token_with_the_tiles_between(N, C, F):
    """Batches whose dx is too little for large tiles and too much for the smallest."""
    x, wg, wu = operands(19, N, C, F)
    _, s = det.gated_linear_forward(x, wg, wu)
    dh = torch.randn(N, F, device=DEV).to(BF16)
    dx = det.gated_linear_backward(dh, x, wg, wu, s, need_dw=False)[0]
    for a, b in ((0, 1), (N - 67, N), (100, 400)):
        cut = det.GatedState(*(type(p)(p[0][a:b], p[1][a:b]) for p in s))
        assert torch.equal(det.gated_linear_backward(dh[a:b], None, wg, wu, cut, need_dw=False)[0], dx[a:b])


@pytest.mark.parametrize("N", [3, 70, 300])
@pytest.mark.parametrize("C", [64, 100, 128])
def test_layouts(N, C):
    F = 65
    x, wg, wu = operands(10, N, C, F)
    h, s = det.gated_linear_forward(x, wg, wu)
    dh = torch.randn(N, F, device=DEV).to(BF16)
    want = det.gated_linear_backward(dh, x, wg, wu, s)
    room = lambda t, off, pad: torch.zeros(t.shape[0], t.shape[1] + pad, device=DEV, dtype=t.dtype)[:, off:off + t.shape[1]].copy_(t)
    views = [(room(x, 1, 3), room(wg, 8, 16), room(wu, 2, 2)), (room(x, 8, 8), room(wg, 0, 8), wu),
             (x.t().contiguous().t(), wg.t().contiguous().t(), room(wu, 8, 24))]
    for v in views:
        h2, s2 = det.gated_linear_forward(*v)
        assert torch.equal(h2, h) and torch.equal(det.gated_linear(*v), h)
        for d in (dh, room(dh, 3, 4), dh.t().contiguous().t()):
            for a, b in zip(det.gated_linear_backward(d, *v, s2), want):
                assert torch.equal(a, b)
    # one row repeated, leading dimensions, a gradient that is one value
    e = x[:1].expand(N, C)
    assert torch.equal(det.gated_linear(e, wg, wu), det.gated_linear(x[:1], wg, wu).expand(N, F))
    x3 = x.reshape(N, 1, C).requires_grad_(True)
    y = det.gated_linear(x3, wg, wu)
    assert y.shape == (N, 1, F)
    gx, = torch.autograd.grad(y.sum(), x3)
    assert torch.equal(gx.reshape(N, C), det.gated_linear_backward(torch.ones_like(h), x, wg, wu, s, need_dw=False)[0])


def test_one_feature_of_wider_weights():
    """Weights of one row each, whose strides are whatever their slices left."""
    x, wg, wu = operands(18, 70, 64, 8)
    ones = wg[::8], wu[:1]
    assert ones[0].stride(0) != ones[1].stride(0) and all(w.is_contiguous() for w in ones)
    h, s = det.gated_linear_forward(x, *ones)
    want_h, want_s = det.gated_linear_forward(x, wg[:1].clone(), wu[:1].clone())
    dh = torch.ones_like(h)
    assert torch.equal(h, want_h)
    for a, b in zip(det.gated_linear_backward(dh, x, *ones, s),
                    det.gated_linear_backward(dh, x, wg[:1].clone(), wu[:1].clone(), want_s)):
        assert torch.equal(a, b)


def test_no_rows():
    x, wg, wu = operands(11, 4, 40, 24)
    x = x[:0].requires_grad_(True)
    for ck in (None, "int8"):
        w = wg.clone().requires_grad_(True)
        h = det.gated_linear(x, w, wu, checkpoint=ck)
        assert h.shape == (0, 24)
        gx, gw = torch.autograd.grad(h, (x, w), torch.empty_like(h))
        assert gx.shape == (0, 40) and torch.equal(gw, torch.zeros_like(w))


@pytest.mark.parametrize("N", [63, 129, 1000, 4097])
@pytest.mark.parametrize("C,F", [(64, 30), (100, 300), (130, 1000)])
def test_weight_gradients_over_long_batches_of_narrow_layers(N, C, F):
    """Few tiles and a long chain.  Integers: all sums are exact, whatever lies past the last row."""
    g = torch.Generator(device=DEV).manual_seed(20)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).to(BF16)
    x = ints(N + 300, C)
    x[N:] = float("inf")                                # rows of the batch that this call is not given
    x = x[:N]
    wg, wu = torch.zeros(2, F, C, device=DEV, dtype=BF16)
    wg[:, 0] = wu[:, 0] = 1.0
    _, s = det.gated_linear_forward(x, wg, wu)
    dh = ints(N, F)
    gates = det.GatedState(det.ScaledHalf(torch.zeros_like(s.gate[0]), s.gate[1]), s.up)
    # g = 0: silu is 0 and its slope 1/2, so dg = dh u / 2 and du = 0
    _, dwg, dwu = det.gated_linear_backward(dh, x, wg, wu, gates, need_dx=False)
    dg = (dh.double() * x[:, :1].double() / 2).to(BF16).double()
    want = dg.t() @ x.double()
    assert want.abs().max() < 2 ** 24 and torch.equal(dwg, want.to(torch.float32).to(BF16))
    assert torch.equal(dwu, torch.zeros_like(dwu))


def test_rows_that_are_not_finite_stay_by_themselves():
    x, wg, wu = operands(12, 200, 96, 130)
    clean, s0 = det.gated_linear_forward(x, wg, wu, out_dtype=F32, checkpoint="int8")
    bad = x.clone()
    bad[3, 5], bad[70, 0], bad[199, 95] = float("nan"), float("inf"), -float("inf")
    rows = torch.ones(200, dtype=torch.bool, device=DEV)
    rows[[3, 70, 199]] = False
    h, s = det.gated_linear_forward(bad, wg, wu, out_dtype=F32, checkpoint="int8")
    assert torch.equal(h[rows], clean[rows]) and torch.isnan(h[3]).all() and not torch.isfinite(h[70]).any()
    assert torch.equal(s.gate.codes[rows], s0.gate.codes[rows])
    assert (s.gate.exponents[~rows] == -128).all() and (s.up.exponents[~rows] == -128).all()
    # in 16 bits an element that is not finite stays by itself
    wide = wg.clone()
    wide[7] = float("inf")
    kept = det.gated_linear_forward(x, wide, wu)[1]
    fine = det.gated_linear_forward(x, wg, wu)[1]
    cols = torch.arange(130, device=DEV) != 7
    assert not torch.isfinite(value(kept.gate)[:, 7]).any()
    assert ((value(kept.gate) - value(fine.gate)).abs()[:, cols] <= 2.0 ** -10 * value(fine.gate).abs()[:, cols]).all()
    # sizes that fp16 alone would lose
    for scale in (2.0 ** 40, 2.0 ** -60):
        big = det.gated_linear_forward((x.double() * scale).to(BF16), wg, wu)[1]
        assert torch.equal(big.gate.values, fine.gate.values)
    # large arguments: the activations reach their limits
    wide = torch.full((70, 1), 3.0e4, device=DEV, dtype=BF16)
    one = torch.ones(8, 1, device=DEV, dtype=BF16)
    for act in ACTS:
        assert torch.equal(det.gated_linear(wide, one, one, activation=act), (wide * wide).expand(70, 8).to(BF16))
        low = det.gated_linear(wide, -one, one, activation=act)
        assert (low == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    # f = sum(dh h) along a direction of each input; h has 32 bits, the inputs move by what bf16 holds exactly
    N, C, F = 24, 48, 40
    g = torch.Generator(device=DEV).manual_seed(13)
    leaves = [(integers(g, *s, top=4).double() / 8).to(BF16).requires_grad_(True) for s in ((N, C), (F, C), (F, C))]
    dh = torch.randn(N, F, device=DEV, generator=g)
    grads = torch.autograd.grad(det.gated_linear(*leaves, activation=act, out_dtype=F32), leaves, dh)
    step = 2.0 ** -6
    for i, t in enumerate(leaves):
        d = integers(g, *t.shape, top=1)
        f = []
        for sign in (1, -1):
            moved = [l.detach() if j != i else (l.detach().double() + sign * step * d.double()).to(BF16) for j, l in enumerate(leaves)]
            assert all(torch.equal((l.detach().double() + sign * step * d.double()), m.double()) for j, (l, m) in enumerate(zip(leaves, moved)) if j == i)
            f.append((det.gated_linear(*moved, activation=act, out_dtype=F32).double() * dh.double()).sum())
        slope = (f[0] - f[1]) / (2 * step)
        want = (grads[i].double() * d.double()).sum()
        # third derivatives along d: |d|^3 terms of size step^2 / 6; roundings of the gradient's elements
        noise = 2 * U[BF16] * (grads[i].double() * d.double()).norm() * 4 + step ** 2 * dh.double().abs().sum() * 8
        assert abs(slope - want) <= noise, (i, slope.item(), want.item(), noise.item())


def test_streams_and_graphs():
    x, wg, wu = operands(14, 300, 100, 70)
    dh = torch.randn(300, 70, device=DEV).to(BF16)
    for ck in (None, "int8"):
        def step(x, wg, wu, dh):
            h, s = det.gated_linear_forward(x, wg, wu, checkpoint=ck)
            kx = det.pack_int8(x) if ck else x
            return (h, det.gated_linear(x[:20], wg, wu), *det.gated_linear_backward(dh, kx, wg, wu, s))
        want = step(x, wg, wu, dh)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step(x, wg, wu, dh)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # leaves made for the capture, replayed on new data with eager work between
        bufs = [t.clone() for t in (x, wg, wu, dh)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step(*bufs)
        for k in range(3):
            fresh = operands(20 + k, 300, 100, 70)
            for b, t in zip(bufs, fresh):
                b.copy_(t)
            graph.replay()
            eager = step(*bufs)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, eager))


def test_second_derivatives_are_refused():
    x, wg, wu = operands(15, 20, 32, 16)
    for ck in (None, "int8"):
        for i in range(3):
            leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, wg, wu))]
            h = det.gated_linear(*leaves, checkpoint=ck, out_dtype=F32)
            g, = torch.autograd.grad(h.sum(), leaves[i], create_graph=True)
            with pytest.raises(RuntimeError, match="differentiable once"):
                torch.autograd.grad(g.float().square().sum(), leaves[i])


def test_module_and_a_feed_forward_block():
    torch.manual_seed(0)
    up = det.DetGatedLinear(96, 200, activation="gelu_tanh", device=DEV, checkpoint="int8")
    down = det.DetLinear(200, 96, device=DEV, dtype=BF16)
    x = torch.randn(2, 50, 96, device=DEV).to(BF16).requires_grad_(True)
    y = down(up(x))
    assert y.shape == (2, 50, 96) and y.dtype == F32
    grads = torch.autograd.grad(det.exact_mse_loss(y), [x, *up.parameters(), *down.parameters()])
    assert all(torch.isfinite(g).all() and g.dtype == BF16 for g in grads)
    again = torch.autograd.grad(det.exact_mse_loss(down(up(x))), [x, *up.parameters(), *down.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("ck", [None, "int8"])
def test_frozen_weights_keep_nothing_of_x(ck):
    x, wg, wu = operands(17, 70, 100, 65)
    dh = torch.randn(70, 65, device=DEV).to(BF16)
    _, s = det.gated_linear_forward(x, wg, wu, checkpoint=ck)
    x.requires_grad_(True)
    sizes = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append(tuple(t.shape)), t)[1], lambda t: t):
        h = det.gated_linear(x, wg, wu, checkpoint=ck)
    assert (70, 100) not in sizes and (70, 4) not in sizes
    dx, = torch.autograd.grad(h, x, dh)
    assert torch.equal(dx, det.gated_linear_backward(dh, None, wg, wu, s, need_dw=False)[0])
    # one weight alone, no gradient of x
    for i in (1, 2):
        leaves = [t.detach().clone().requires_grad_(j == i) for j, t in enumerate((x, wg, wu))]
        kx = det.pack_int8(x) if ck else x.detach()
        g, = torch.autograd.grad(det.gated_linear(*leaves, checkpoint=ck), leaves[i], dh)
        assert torch.equal(g, det.gated_linear_backward(dh, kx, wg, wu, s, need_dx=False)[i])


@pytest.mark.parametrize("N,F", [(70, 40), (300, 130)])
def test_rows_far_apart(N, F):
    # strides up to the largest that is read in place (2^21 elements), and above it
    C = 64
    x, wg, wu = operands(18, N, C, F)
    dh = torch.randn(N, F, device=DEV).to(BF16)
    h, s = det.gated_linear_forward(x, wg, wu)
    want = det.gated_linear_backward(dh, x, wg, wu, s)
    for stride in (1 << 21, (1 << 21) + 8, 1 << 22):
        room = torch.empty(max(N, F) * stride, dtype=BF16, device=DEV)
        far = lambda t: room.as_strided(t.shape, (stride, 1)).copy_(t)
        for i in range(3):
            v = [far(t) if j == i else t for j, t in enumerate((x, wg, wu))]
            h2, s2 = det.gated_linear_forward(*v)
            assert torch.equal(h2, h)
            assert all(torch.equal(a, b) for a, b in zip(det.gated_linear_backward(dh, *v, s2), want))
        del room


@pytest.mark.parametrize("N", [1, 70])
def test_gelu_against_64_bits(N):
    """Any fp32 value as g, from three bf16 parts, times u = 1."""
    r = 1e-6 * 1.3e7 ** torch.rand(8192, device=DEV, dtype=torch.float64, generator=torch.Generator(device=DEV).manual_seed(21))
    g = torch.cat([r, -r]).float()
    hi = g.to(BF16)
    mid = (g - hi.float()).to(BF16)
    lo = (g - hi.float() - mid.float()).to(BF16)
    zero, one = torch.zeros_like(hi), torch.ones_like(hi)
    wg, wu = torch.stack([hi, mid, lo, zero], 1), torch.stack([one, zero, zero, zero], 1)
    x = torch.tensor([1, 1, 1, 0], device=DEV, dtype=BF16).expand(N, 4)
    h = det.gated_linear(x, wg, wu, activation="gelu", out_dtype=F32)
    G = hi.double() + mid.double() + lo.double()
    want = G * 0.5 * torch.special.erfc(-G / math.sqrt(2.0))
    # half steps: 4 of the exponential and 1 of its correction, 3 of the polynomial, 2 of the reciprocal, 1 of the fit,
    # 5 products and the difference from 1; g itself is a sum of three parts in 32 bits (2, and g Phi(g) changes by up to
    # (1 + g^2) times as much below 0)
    bound = (16 + 2 * (1 + G * G)) * U[F32] * want.abs() + 1e-37
    for row in h:
        within(row, want, bound, "gelu")


def test_activations_far_out():
    # their limits' slopes, 1 and 0, as far as fp32 goes
    one = torch.ones(70, 1, device=DEV, dtype=BF16)
    for act in ACTS:
        for size in (1e3, 1e10, 1e20, 1e30):
            for sign in (1.0, -1.0):
                wg, wu = torch.full((8, 1), sign * size, device=DEV, dtype=BF16), torch.full((8, 1), 2.0 ** -60, device=DEV, dtype=BF16)
                h, s = det.gated_linear_forward(one, wg, wu, activation=act)
                dx, dwg, dwu = det.gated_linear_backward(torch.ones(70, 8, device=DEV, dtype=BF16), one, wg, wu, s, activation=act)
                assert torch.isfinite(dx).all()
                g, u = wg[0, 0].item(), 2.0 ** -60
                assert dwg[0, 0].item() == (70 * u if sign > 0 else 0)
                assert abs(dwu[0, 0].item() - (70 * g if sign > 0 else 0)) <= 2 * U[BF16] * abs(70 * g)


def test_rows_past_32_bits():
    # h, what is kept and dg and du pass 2^32 bytes; the last rows are those of a small batch
    N, C, F = 560000, 64, 4160
    g = torch.Generator(device=DEV).manual_seed(16)
    x = torch.randn(N, C, generator=g, device=DEV).to(BF16)
    wg, wu = (torch.randn(F, C, generator=g, device=DEV).to(BF16) / 8 for _ in range(2))
    h, s = det.gated_linear_forward(x, wg, wu)
    part, t = det.gated_linear_forward(x[-70:], wg, wu)
    assert torch.equal(h[-70:], part) and torch.equal(s.up.values[-70:], t.up.values)
    assert torch.equal(s.gate.exponents[-70:], t.gate.exponents)
    # a gradient of the last rows alone: dx is theirs, dw is that of these rows after rows of zeros
    dh = torch.zeros(N, F, device=DEV, dtype=BF16)
    dh[-64:] = torch.randn(64, F, generator=g, device=DEV).to(BF16)
    dx, dwg, dwu = det.gated_linear_backward(dh, x, wg, wu, s)
    small = det.gated_linear_backward(dh[-64:], x[-64:], wg, wu, det.gated_linear_forward(x[-64:], wg, wu)[1])
    assert torch.equal(dx[-64:], small[0]) and (dx[:-64] == 0).all()
    assert torch.equal(dwg, small[1]) and torch.equal(dwu, small[2])
