"""The gated projection's largest tiles, which carry prompts and large training
steps: 256 x 256 and 128 x 256 outputs, ragged both ways and on widths that are
padded, with every kind of kept projections, and products in two launches.  And what a call notes and copies beside its products."""
import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests import test_gpu_gated as base
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32

# forward in tiles of 256 x 256 and dw of 128 x 256; forward of 128 x 256 and dw of 256 x 256; dx of 128 x 256, forward and dw of
# 256 x 256; dx of 256 x 256; two launches, the second with smaller tiles: of the forward's features, of its rows, of dx' columns,
# of its rows
SIZES = [(2000, 1023, 2801), (1100, 2100, 2817), (3000, 2112, 2112), (8200, 1030, 260), (1021, 1537, 4099), (5000, 1100, 1000),
         (4100, 2100, 700), (2050, 2111, 1100)]


@pytest.mark.parametrize("N,C,F", SIZES)
def test_products_are_exact_on_integers(N, C, F):
    base.test_products_are_exact_on_integers(N, C, F)


@pytest.mark.parametrize("act,out", [("silu", BF16), ("gelu", F32)])
@pytest.mark.parametrize("N,C,F", SIZES)
def test_forward_against_64_bits(N, C, F, act, out):
    base.test_forward_against_64_bits(N, C, F, act, out)


@pytest.mark.parametrize("act,dtype", [("silu", F32), ("gelu_tanh", BF16)])
@pytest.mark.parametrize("N,C,F", SIZES)
def test_gradients_against_64_bits(N, C, F, act, dtype):
    base.test_gradients_against_64_bits(N, C, F, act, dtype)


@pytest.mark.parametrize("N,C,F", SIZES)
def test_int8_checkpoint(N, C, F):
    base.test_int8_checkpoint(N, C, F)


@pytest.mark.parametrize("N,C,F", SIZES)
def test_a_token_is_the_same_in_any_batch(N, C, F):
    """One token, decode batches and parts of the batch, whose tiles are others: the same bits."""
    announce(f"gated batch {N} {C} {F}")
    x, wg, wu = base.operands(31, N, C, F)
    dh = torch.randn(N, F, device=DEV, generator=torch.Generator(device=DEV).manual_seed(32))
    whole = {ck: det.gated_linear_forward(x, wg, wu, out_dtype=F32, checkpoint=ck) for ck in (None, "int8")}
    dx = {ck: det.gated_linear_backward(dh, None, wg, wu, s, need_dw=False)[0] for ck, (_, s) in whole.items()}
    for a, b in ((0, 1), (N - 1, N), (37, 53), (N - 64, N), (100, 400), (255, N - 255)):
        assert torch.equal(det.gated_linear(x[a:b], wg, wu, out_dtype=F32), whole[None][0][a:b])
        for ck, (h, s) in whole.items():
            part, t = det.gated_linear_forward(x[a:b], wg, wu, out_dtype=F32, checkpoint=ck)
            assert torch.equal(part, h[a:b])
            for p, q in zip(t, s):
                assert torch.equal(p[0], q[0][a:b]) and torch.equal(p[1], q[1][a:b])
            assert torch.equal(det.gated_linear_backward(dh[a:b], None, wg, wu, t, need_dw=False)[0], dx[ck][a:b])


@pytest.mark.parametrize("N,C,F", [(1500, 2112, 5000), (1500, 1600, 6000), (2000, 3000, 4000), (300, 4096, 11008)])
def test_weight_gradients_in_two_launches(N, C, F):
    """On integers every sum is exact: dw = dg^T x with dg = dh u / 2 where g is 0."""
    announce(f"gated two launches {N} {C} {F}")
    g = torch.Generator(device=DEV).manual_seed(33)
    x = base.integers(g, N, C)
    wg, wu = torch.zeros(2, F, C, device=DEV, dtype=BF16)
    wg[:, 0] = wu[:, 0] = 1.0
    _, s = det.gated_linear_forward(x, wg, wu)
    dh = base.integers(g, N, F)
    gates = det.GatedState(det.ScaledHalf(torch.zeros_like(s.gate[0]), s.gate[1]), s.up)
    _, dwg, dwu = det.gated_linear_backward(dh, x, wg, wu, gates, need_dx=False)
    dg = (dh.double() * x[:, :1].double() / 2).to(BF16).double()
    want = dg.t() @ x.double()
    assert want.abs().max() < 2 ** 24 and torch.equal(dwg, want.to(F32).to(BF16))
    assert torch.equal(dwu, torch.zeros_like(dwu))


def test_projections_that_overflow_are_noted():
    """A block of 8 bits that is not finite spoils the gradients of its 32 features: device_status() says so."""
    x, wg, wu = base.operands(34, 70, 64, 100)
    det.device_status()
    det.gated_linear_forward(x, wg, wu, checkpoint="int8")
    assert not det.device_status()
    big = x.clone()
    big[5] = 1e30                                       # finite, and so are the weights
    for i in range(2):
        w = [wg, wu]
        w[i] = w[i].clone()
        w[i][40] = 1e30
        s = det.gated_linear_forward(big, *w, checkpoint="int8")[1]
        assert s[i].exponents[5, 1] == -128 and (s[i].exponents == -128).sum() == 1
        assert "nonfinite" in det.device_status()
        det.gated_linear_forward(big[:5], *w, checkpoint="int8")
        assert not det.device_status()
    # in a tile of 256 x 256, too
    x, wg, wu = base.operands(37, 2000, 1024, 2816)
    for i in range(2):
        w = [wg.clone(), wu.clone()]
        det.gated_linear_forward(x, *w, checkpoint="int8")
        assert not det.device_status()
        w[i][2815, 1023] = float("inf")
        s = det.gated_linear_forward(x, *w, checkpoint="int8")[1]
        assert (s[i].exponents[:, -1] == -128).all() and "nonfinite" in det.device_status()


def bytes_taken(call):
    call()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    out = call()
    return torch.cuda.max_memory_allocated() - before, out


@pytest.mark.parametrize("N", [1, 16, 17, 64])
def test_few_tokens_copy_no_weights(N):
    """Weights that are column slices at odd offsets: 64 tokens at most read them as they lie."""
    C, F = 1024, 3000
    x, wg, wu = base.operands(35, N, C, F)
    want = det.gated_linear(x, wg, wu)
    odd = lambda t: torch.zeros(F, C + 3, device=DEV, dtype=BF16)[:, 1:C + 1].copy_(t)
    g, u = odd(wg), odd(wu)
    for pair in ((g, u), (g, wu), (wg, u)):
        taken, h = bytes_taken(lambda: det.gated_linear(x, *pair))
        assert torch.equal(h, want) and taken < F * C


@pytest.mark.parametrize("ck", [None, "int8"])
def test_weight_gradients_copy_no_weights(ck):
    """The weights' own gradients do not read them: slices and unequal strides stay as they are."""
    N, C, F = 64, 1024, 3000
    x, wg, wu = base.operands(36, N, C, F)
    h, s = det.gated_linear_forward(x, wg, wu, checkpoint=ck)
    want = det.gated_linear_backward(h, x, wg, wu, s)
    room = lambda t, off, pad: torch.zeros(F, C + pad, device=DEV, dtype=BF16)[:, off:off + C].copy_(t)
    outputs = 2 * F * C * 2 + 2 * N * (F + 128) * 2
    for pair in ((room(wg, 1, 3), room(wu, 2, 5)), (wg, room(wu, 8, 16))):
        taken, got = bytes_taken(lambda: det.gated_linear_backward(h, x, *pair, s, need_dx=False))
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]) and taken < outputs + F * C
        assert torch.equal(det.gated_linear_backward(h, x, *pair, s)[0], want[0])
