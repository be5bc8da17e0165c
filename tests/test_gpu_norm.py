"""Layer norm on the GPU against the formulas in 64 bits, at widths and row
counts on both sides of every kernel boundary, in every mix of types; the
exactness of the weights' gradients over rows, and their composition over row
shards.

Tolerances, derived before the first run.  u = 2^-24 (an fp32 rounding).  A
row's sums add at most 32 values per thread one after another and then at most
6 + 16 more, so a sum of n terms t is within 56 u sum|t| (each term itself
rounded at most twice); the mean is corrected once, the variance, root and
division add 4 u.  That puts h within 64 u (1 + |h|), y within 64 u (1 +
|h|)|w| + 2 u (|h w| + |b|).  The backward pass reads the mean rounded to
fp32, which moves h by at most u |mean| rstd more.  A result's own rounding
adds half a step of its type, eps / 2 of the value.
"""
import math

import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
NAMES = {F32: "f32", BF16: "bf16"}
# widths around every register geometry (512, 1024, 2048, ...), odd ones, one
# element, the widest; rows around the chunks of 16 and 32
SIZES = [(1, 1), (3, 2), (5, 7), (17, 511), (16, 512), (33, 513), (31, 1024), (65, 1025), (32, 2048), (64, 2049),
         (34, 4095), (1, 4096), (100, 4097), (7, 8192), (33, 8193), (3, 16384), (35, 16385), (2, 32767), (3, 32768),
         (1500, 96), (2500, 33)]


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def _inputs(N, C, xt, wt, yt, seed, offset=0.0, weights=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, C, generator=g) * 1.5 + offset).to(xt)
    w = (1 + 0.2 * torch.randn(C, generator=g)).to(wt) if weights else None
    b = (0.3 * torch.randn(C, generator=g)).to(wt) if weights else None
    dy = torch.randn(N, C, generator=g).to(yt)
    return x.cuda(), None if w is None else w.cuda(), None if b is None else b.cuda(), dy.cuda()


def _formula(x, w, b, dy, eps):
    """y, h, dx, dw, db and the row quantities in 64 bits."""
    X, DY = x.double(), dy.double()
    W = w.double() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64, device=x.device)
    Bb = b.double() if b is not None else torch.zeros_like(W)
    mean = X.mean(-1, keepdim=True)
    d = X - mean
    r = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    h = d * r
    g = DY * W
    dx = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return dict(y=h * W + Bb, h=h, r=r, mean=mean, g=g, dx=dx, dw=(DY * h).sum(0), db=DY.sum(0), W=W, B=Bb, DY=DY)


def _check(name, got, want, tol):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), name
    bad = err > tol
    assert not bad.any(), f"{name}: {int(bad.sum())} beyond tolerance, worst ratio {(err / tol).max().item():.3g}"


def _check_forward(y, q, out_dtype):
    h, W, Bb = q["h"].abs(), q["W"].abs(), q["B"].abs()
    tol = 64 * U * (1 + h) * W + 2 * U * (h * W + Bb)
    _check("y", y, q["y"], tol + half_step(out_dtype) * (q["y"].abs() + tol))


def _check_backward(dx, dw, db, q, xt, wt):
    h, g, r = q["h"].abs(), q["g"].abs(), q["r"]
    dh = 64 * U * (1 + h) + U * q["mean"].abs() * r                 # of the recomputed h
    m1 = g.mean(-1, keepdim=True)
    m2 = (g * h).mean(-1, keepdim=True)
    tol = r * (4 * U * g + 64 * U * m1 + (dh + 4 * U * h) * m2 + h * (64 * U * m2 + (g * dh).mean(-1, keepdim=True)))
    tol = tol + 4 * U * q["dx"].abs()
    _check("dx", dx, q["dx"], tol + half_step(xt) * (q["dx"].abs() + tol))
    dy = q["DY"].abs()
    # at most 64 rows added in fp32 (8 groups of 8), the rest exactly
    for name, got, want, t in (("dw", dw, q["dw"], (dy * (dh + 36 * U * h)).sum(0)),
                               ("db", db, q["db"], (36 * U * dy).sum(0))):
        t = t + 2.0 ** -149
        _check(name, got, want, t + U * want.abs() + half_step(wt) * (want.abs() + t))


@pytest.mark.parametrize("N,C", SIZES)
@pytest.mark.parametrize("types", [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, BF16), (BF16, F32, F32)],
                         ids=lambda t: "-".join(NAMES[v] for v in t))
def test_forward_and_backward(N, C, types):
    xt, wt, yt = types
    announce(f"layer norm {N}x{C} x={NAMES[xt]} w={NAMES[wt]} y={NAMES[yt]}")
    x, w, b, dy = _inputs(N, C, xt, wt, yt, 1000 * N + C)
    q = _formula(x, w, b, dy, 1e-5)
    y, mean, rstd = det.layer_norm_forward(x, w, b, 1e-5, yt)
    assert y.dtype == yt and mean.shape == rstd.shape == (N,)
    if C > 1:                                                       # C = 1: h = 0 exactly
        _check_forward(y, q, yt)
    else:
        assert torch.equal(y, b.to(yt).expand(N, 1))
    dx, dw, db = det.layer_norm_backward(dy, x, w, mean, rstd)
    assert dx.dtype == xt and dw.dtype == db.dtype == wt
    _check_backward(dx, dw, db, q, xt, wt)
    # autograd gives the same bits
    xr, wr, br = (t.clone().requires_grad_(True) for t in (x, w, b))
    ya = det.layer_norm(xr, wr, br, 1e-5, yt)
    ga = torch.autograd.grad(ya, (xr, wr, br), dy)
    assert torch.equal(ya, y) and all(torch.equal(p, q_) for p, q_ in zip(ga, (dx, dw, db)))


@pytest.mark.parametrize("offset", [1000.0, -3.0e4])
def test_offset_rows_keep_their_precision(offset):
    # |mean| far above the spread: the plain one-pass variance would lose everything
    x, w, b, dy = _inputs(40, 1000, F32, F32, F32, 5, offset)
    q = _formula(x, w, b, dy, 1e-5)
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    _check_forward(y, q, F32)
    _check_backward(*det.layer_norm_backward(dy, x, w, mean, rstd), q, F32, F32)


def test_constant_rows_and_eps():
    # zero variance: h = 0 (x exactly representable), rstd = 1 / sqrt(eps)
    x = torch.full((9, 300), 2.5, device="cuda")
    b = torch.randn(300, device="cuda")
    y, mean, rstd = det.layer_norm_forward(x, None, b, 1e-4)
    assert torch.equal(y, b.expand(9, 300)) and torch.equal(mean, torch.full((9,), 2.5, device="cuda"))
    assert torch.allclose(rstd, torch.full((9,), 100.0, device="cuda"), rtol=4 * U * 4, atol=0)


@pytest.mark.parametrize("C", [33, 4096])
def test_optional_weights_and_needs(C):
    x, w, b, dy = _inputs(50, C, F32, F32, F32, 8)
    for ww, bb in ((None, None), (w, None), (None, b)):
        q = _formula(x, ww, bb, dy, 1e-5)
        y, mean, rstd = det.layer_norm_forward(x, ww, bb)
        _check_forward(y, q, F32)
        full = det.layer_norm_backward(dy, x, ww, mean, rstd)
        _check_backward(*full, q, F32, F32)
        for needs in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
            got = det.layer_norm_backward(dy, x, ww, mean, rstd, need_dx=needs[0], need_dweight=needs[1],
                                          need_dbias=needs[2])
            for g, f, n in zip(got, full, needs):
                assert (g is None) if not n else torch.equal(g, f)
        # through autograd, with the absent weights' places empty
        leaves = [t.clone().requires_grad_(True) if t is not None else None for t in (x, ww, bb)]
        grads = torch.autograd.grad(det.layer_norm(*leaves), [t for t in leaves if t is not None], dy)
        assert all(torch.equal(p, f) for p, f in zip(grads, [f for f, t in zip(full, leaves) if t is not None]))


def test_leading_shapes_strides_and_broadcast_gradients():
    x, w, b, _ = _inputs(6 * 7, 130, BF16, F32, F32, 9)
    base, mean, rstd = det.layer_norm_forward(x, w, b, out_dtype=F32)
    assert torch.equal(det.layer_norm(x.reshape(6, 7, 130), w, b, out_dtype=F32), base.reshape(6, 7, 130))
    assert det.layer_norm(x[0], w, b, out_dtype=F32).shape == (130,)
    assert torch.equal(det.layer_norm(x[0], w, b, out_dtype=F32), base[0])
    # rows apart and misaligned, a transposed view, rows repeated with stride 0
    wide = torch.zeros(42, 199, dtype=BF16, device="cuda")
    wide[:, 3:133] = x
    assert torch.equal(det.layer_norm(wide[:, 3:133], w, b, out_dtype=F32), base)
    assert torch.equal(det.layer_norm(x.t().contiguous().t(), w, b, out_dtype=F32), base)
    assert torch.equal(det.layer_norm(x[:1].expand(42, 130), w, b, out_dtype=F32), base[:1].expand(42, 130))
    # a broadcast incoming gradient (of y.sum()) and a sliced one
    one = torch.ones((), device="cuda").expand(42, 130)
    got = det.layer_norm_backward(one, x, w, mean, rstd)
    want = det.layer_norm_backward(one.contiguous(), x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    dy = torch.randn(42, 140, device="cuda")
    got = det.layer_norm_backward(dy[:, 7:137], x, w, mean, rstd)
    want = det.layer_norm_backward(dy[:, 7:137].contiguous(), x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_no_rows():
    x = torch.empty(0, 40, device="cuda", requires_grad=True)
    w = torch.ones(40, device="cuda", requires_grad=True)
    y = det.layer_norm(x, w)
    assert y.shape == (0, 40)
    dx, dw = torch.autograd.grad(y.sum(), (x, w))
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros(40, device="cuda"))


@pytest.mark.parametrize("C", [100, 1500, 4096])
def test_rows_do_not_depend_on_the_batch(C):
    x, w, b, dy = _inputs(3000, C, BF16, BF16, BF16, 12)
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    dx = det.layer_norm_backward(dy, x, w, mean, rstd)[0]
    for rows in (slice(0, 1), slice(5, 6), slice(2999, 3000), slice(7, 260)):
        y1, m1, r1 = det.layer_norm_forward(x[rows], w, b)
        assert torch.equal(y1, y[rows]) and torch.equal(m1, mean[rows]) and torch.equal(r1, rstd[rows])
        assert torch.equal(det.layer_norm_backward(dy[rows], x[rows], w, m1, r1)[0], dx[rows])


@pytest.mark.parametrize("C,cuts", [(70, (0, 64, 192, 1000, 1001)), (4096, (0, 64, 320, 333))])
def test_row_shards_compose_to_the_same_bits(C, cuts):
    cuts = tuple(c // 64 * 64 for c in cuts[:-1]) + (cuts[-1],)
    N = cuts[-1]
    x, w, b, dy = _inputs(N, C, F32, F32, F32, 21)
    _, mean, rstd = det.layer_norm_forward(x, w, b)
    _, dw, db, digits = det.layer_norm_backward(dy, x, w, mean, rstd, digits=True)
    assert torch.equal(det.det_finalize(digits), torch.stack([dw, db]))
    parts = [det.layer_norm_digits(dy[a:e], x[a:e], mean[a:e], rstd[a:e]) for a, e in zip(cuts, cuts[1:])]
    for order in (parts, parts[::-1], parts[1:] + parts[:1]):
        total = det.det_combine(order)
        assert torch.equal(total, digits)
        assert torch.equal(det.det_finalize(total), torch.stack([dw, db]))


@pytest.mark.parametrize("C", [5, 64])
def test_bias_gradient_adds_chunks_exactly(C):
    # a chunk of huge rows, one of ones, one that cancels the first: any
    # floating-point order over the chunks loses the ones
    x, _, _, _ = _inputs(192, C, F32, F32, F32, 30)
    dy = torch.zeros(192, C, device="cuda")
    dy[0], dy[70], dy[71], dy[150] = 2.0 ** 100, 1.0, 2.0 ** -30, -(2.0 ** 100)
    _, mean, rstd = det.layer_norm_forward(x)
    db = det.layer_norm_backward(dy, x, None, mean, rstd)[2]
    assert torch.equal(db, torch.full((C,), 1.0, device="cuda"))
    dy[71] = 2.0 ** -20
    db = det.layer_norm_backward(dy, x, None, mean, rstd)[2]
    assert torch.equal(db, torch.full((C,), 1.0 + 2.0 ** -20, device="cuda"))


def test_rounding_of_the_chunk_sum():
    # ties, carries, subnormals, overflow and exact zero, each through its own
    # column; the digits rounded by det_finalize give the same bits
    cases = [(1.0, 2.0 ** -24), (1.0 + 2.0 ** -23, 2.0 ** -24), (1.0, 2.0 ** -24 + 2.0 ** -40), (1.0, -2.0 ** -25),
             (2.0 ** -149, 2.0 ** -149), (2.0 ** -126, -2.0 ** -149), (3.0e38, 3.0e38), (-3.0e38, -3.0e38),
             (5.5, -5.5), (-1.0, 2.0 ** -60), (2.0 ** 24 - 1, 0.5), (0.0, -0.0), (2.0 ** -140, 2.0 ** -149 * 3)]
    C = len(cases)
    dy = torch.zeros(100, C, device="cuda")
    dy[0] = torch.tensor([a for a, _ in cases])
    dy[99] = torch.tensor([b for _, b in cases])
    x = torch.randn(100, C, device="cuda")
    _, mean, rstd = det.layer_norm_forward(x)
    _, _, db, digits = det.layer_norm_backward(dy, x, None, mean, rstd, digits=True)
    want = (dy[0].double() + dy[99].double()).cpu().float()          # exact in 64 bits but for (-1, 2^-60)
    want[9] = -1.0
    assert torch.equal(db.cpu(), want)
    assert torch.equal(det.det_finalize(digits)[1].cpu(), want)


def test_many_rows_split_the_columns():
    # enough chunks that several workgroups share a column
    x, w, b, dy = _inputs(40000, 24, F32, F32, F32, 33)
    q = _formula(x, w, b, dy, 1e-5)
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    dx, dw, db, digits = det.layer_norm_backward(dy, x, w, mean, rstd, digits=True)
    _check_forward(y, q, F32)
    _check_backward(dx, dw, db, q, F32, F32)
    assert torch.equal(det.det_finalize(digits), torch.stack([dw, db]))
    halves = [det.layer_norm_digits(dy[s], x[s], mean[s], rstd[s]) for s in (slice(0, 19200), slice(19200, 40000))]
    assert torch.equal(det.det_combine(halves), digits)


def test_nonfinite_values():
    det.device_status()
    x, w, b, dy = _inputs(70, 40, F32, F32, F32, 34)
    x[3, 5], x[50, 0] = float("nan"), float("inf")
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[3] = bad[50] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    dx, dw, db = det.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[~bad]).all()
    assert torch.isnan(dw).all() and torch.isfinite(db).all()
    assert det.device_status() == {"nonfinite"}


def test_gradient_against_differences():
    # central differences of the forward pass in 64 bits along random directions
    x, w, b, dy = _inputs(20, 77, F32, F32, F32, 35)
    _, mean, rstd = det.layer_norm_forward(x, w, b)
    grads = det.layer_norm_backward(dy, x, w, mean, rstd)
    f = lambda X, W, B: (_formula(X, W, B, dy, 1e-5)["y"] * dy.double()).sum()      # noqa: E731
    args = [t.double() for t in (x, w, b)]
    e = 2.0 ** -12
    for i, grad in enumerate(grads):
        v = torch.randn_like(args[i])
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + e * v, args[i] - e * v
        slope = (f(*up) - f(*dn)) / (2 * e)
        want = (grad.double() * v).sum()
        # e^2 truncation, and the fp32 gradient's 64 u of each term
        tol = 4 * e * e * (grad.double().abs() * v.abs()).sum() + 256 * U * (grad.double().abs() * v.abs()).sum()
        assert (slope - want).abs() <= tol, (i, slope, want)


def test_streams_repetition_and_graph_replay():
    x, w, b, dy = _inputs(200, 1030, BF16, F32, BF16, 36)
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    want = det.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            y2, m2, r2 = det.layer_norm_forward(x, w, b)
            got = det.layer_norm_backward(dy, x, w, m2, r2)
            assert torch.equal(y2, y) and all(torch.equal(p, q) for p, q in zip(got, want))
    s.synchronize()
    sx, sdy = x.clone(), dy.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        gy, gm, gr = det.layer_norm_forward(sx, w, b)
        gg = det.layer_norm_backward(sdy, sx, w, gm, gr)
    for k in range(4):
        nx = (x.float() * (k + 1) + k).to(BF16)
        sx.copy_(nx)
        sdy.copy_(dy * (k + 1))
        g.replay()
        torch.cuda.synchronize()
        ey, em, er = det.layer_norm_forward(nx, w, b)
        eg = det.layer_norm_backward(dy * (k + 1), nx, w, em, er)
        assert torch.equal(gy, ey) and all(torch.equal(p, q) for p, q in zip(gg, eg)), k


def test_second_derivatives_are_refused():
    x = torch.randn(3, 20, device="cuda", requires_grad=True)
    dy = torch.randn(3, 20, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(det.layer_norm(x), x, dy, create_graph=True)
    assert torch.equal(g.detach(), torch.autograd.grad(det.layer_norm(x), x, dy)[0])
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.sum().backward()


def test_module_trains():
    m = det.DetLayerNorm(64, device="cuda", dtype=BF16, out_dtype=BF16)
    lin = det.DetLinear(64, 32, device="cuda", dtype=BF16)
    x = torch.randn(4, 9, 64, device="cuda", requires_grad=True)
    lin(m(x)).square().mean().backward()
    assert x.grad.shape == x.shape and m.weight.grad.dtype == BF16 and m.bias.grad.shape == (64,)
    assert math.isfinite(m.weight.grad.float().sum().item())


# Several rows to a wave: each power of two of its lanes and both sides of it,
# rows of less than a vector; row counts around the chunk of 64, and so many
# that workgroups take several rows in turn.  A lane adds at most 8 values and
# a row 5 sums of lanes; a chunk's 64 rows are added within 7 + 7 + 8: the
# bounds above hold as they are.
@pytest.mark.parametrize("C", [2, 4, 6, 8, 9, 15, 16, 17, 31, 32, 40, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257])
@pytest.mark.parametrize("types", [(F32, BF16, F32), (BF16, BF16, BF16), (F32, F32, BF16)],
                         ids=lambda t: "-".join(NAMES[v] for v in t))
def test_short_rows(C, types):
    xt, wt, yt = types
    for N in (1, 63, 130, 2 * 2048 * 256 // min(C, 256) + 5):
        announce(f"layer norm of short rows {N}x{C} x={NAMES[xt]} w={NAMES[wt]} y={NAMES[yt]}")
        x, w, b, dy = _inputs(N, C, xt, wt, yt, 77 * N + C)
        q = _formula(x, w, b, dy, 1e-5)
        y, mean, rstd = det.layer_norm_forward(x, w, b, 1e-5, yt)
        _check_forward(y, q, yt)
        dx, dw, db = det.layer_norm_backward(dy, x, w, mean, rstd)
        _check_backward(dx, dw, db, q, xt, wt)


@pytest.mark.parametrize("C", [3, 24, 128, 250])
def test_short_rows_of_a_wider_tensor_keep_their_bits(C):
    # one row, a part of the rows, rows that are columns of a wider tensor
    x, w, b, dy = _inputs(700, C, BF16, BF16, BF16, 90)
    wide = torch.zeros(700, C + 5, dtype=BF16, device="cuda")
    wide[:, 3:C + 3] = x
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    dx, dw, db = det.layer_norm_backward(dy, x, w, mean, rstd)
    xs = wide[:, 3:C + 3]
    ys, ms, rs = det.layer_norm_forward(xs, w, b)
    assert torch.equal(ys, y) and torch.equal(ms, mean) and torch.equal(rs, rstd)
    assert all(torch.equal(p, q) for p, q in zip(det.layer_norm_backward(dy, xs, w, ms, rs), (dx, dw, db)))
    for rows in (slice(0, 1), slice(699, 700), slice(65, 66), slice(3, 450)):
        y1, m1, r1 = det.layer_norm_forward(x[rows], w, b)
        assert torch.equal(y1, y[rows]) and torch.equal(m1, mean[rows]) and torch.equal(r1, rstd[rows])
        assert torch.equal(det.layer_norm_backward(dy[rows], x[rows], w, m1, r1)[0], dx[rows])


def test_short_rows_keep_nan_and_infinity_to_themselves():
    x, w, b, dy = _inputs(130, 40, F32, F32, F32, 91)
    y, mean, rstd = det.layer_norm_forward(x, w, b)
    dx = det.layer_norm_backward(dy, x, w, mean, rstd)[0]
    x[7, 3], x[8, 0] = float("nan"), float("inf")
    y1, m1, r1 = det.layer_norm_forward(x, w, b)
    dx1 = det.layer_norm_backward(dy, x, w, m1, r1)[0]
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    bad[7:9] = True
    assert torch.equal(y1[~bad], y[~bad]) and torch.equal(dx1[~bad], dx[~bad])
    assert torch.isnan(y1[bad]).all() and torch.isnan(dx1[bad]).all()
