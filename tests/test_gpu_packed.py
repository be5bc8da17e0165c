"""8-bit checkpoints on the GPU: codes and exponents bit for bit against the
format's definition in 64 bits."""
import pytest
import torch

import bitwise_deterministic_exact_amd as det
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def reference(x):
    """(codes, exponents, values) by the definition, on the CPU in 64 bits."""
    x = x.detach().cpu().double()
    lead, C = x.shape[:-1], x.shape[-1]
    b = torch.zeros(*lead, (C + 31) // 32 * 32, dtype=torch.float64)
    b[..., :C] = x
    b = b.unflatten(-1, (-1, 32))
    A = b.abs().amax(-1)
    e = torch.full(A.shape, -126)
    for k in range(-126, 121):              # the least with A < 127.5 2^e, by search
        e += ((e == k) & (A >= 127.5 * 2.0 ** k)).long()
    unit = torch.tensor([2.0 ** k for k in range(-126, 122)], dtype=torch.float64)[e + 126]
    codes = (b / unit[..., None]).round().clamp(-127, 127)
    bad = ~torch.isfinite(b).all(-1)
    codes = torch.where(bad[..., None], 0.0, codes)
    values = torch.where(bad[..., None], float("nan"), codes * unit[..., None]).flatten(-2)[..., :C]
    return codes.flatten(-2)[..., :C].to(torch.int8), torch.where(bad, -128, e).to(torch.int8), values


def check(x):
    p = det.pack_int8(x)
    codes, exps, values = reference(x)
    assert torch.equal(p.codes.cpu(), codes) and torch.equal(p.exponents.cpu(), exps)
    for dt in (F32, BF16):
        y = det.unpack_int8(p, dt)
        assert y.dtype == dt and y.shape == x.shape
        assert torch.equal(torch.nan_to_num(y.cpu().double(), nan=12345.0), torch.nan_to_num(values, nan=12345.0))
    return p


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 8), (1, 32), (4, 33), (7, 31), (2, 3, 64), (100, 1000), (1, 5000),
                                   (9, 1021), (70, 4096), (0, 5), (513,)])
def test_against_the_definition(shape, dtype):
    announce(f"pack {shape} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(shape, generator=g, device=DEV) * torch.exp(3.0 * torch.randn(shape, generator=g, device=DEV))
    check(x.to(dtype))


def test_borders_of_the_exponents():
    top = torch.finfo(F32).max
    rows = []
    for A in (127.0, 127.25, 127.4999, 127.5, 127.75, 128.0, 63.75, 63.7, 1e-37, 2.0 ** -126, 2.0 ** -149, 2.0 ** -127,
              127.5 * 2.0 ** -126, 127.4 * 2.0 ** -126, 2.0 ** 127, 127.5 * 2.0 ** 121, top, 0.0):
        r = torch.linspace(-1, 1, 32, dtype=torch.float64) * A
        r[5] = A
        rows.append(r)
    x = torch.stack(rows).float()
    x[-1, 3] = -0.0
    check(x.to(DEV))
    p = check(x.to(BF16).to(DEV))
    assert torch.isfinite(det.unpack_int8(p)[:-2]).all()


def test_ties_go_to_even():
    x = torch.cat([torch.arange(-8, 8) + 0.5, torch.full((16,), 100.0)]).float()
    p = check(x.to(DEV))
    assert p.exponents.item() == 0 and p.codes[:16].tolist() == [-8, -6, -6, -4, -4, -2, -2, 0, 0, 2, 2, 4, 4, 6, 6, 8]


def test_blocks_that_are_not_finite():
    det.device_status()
    x = torch.randn(6, 100, device=DEV)
    check(x)
    assert not det.device_status()
    x[1, 40], x[2, 99], x[4, 0] = float("nan"), float("inf"), -float("inf")
    p = check(x)
    assert "nonfinite" in det.device_status()
    assert (p.exponents == -128).nonzero().tolist() == [[1, 1], [2, 3], [4, 0]]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layouts(dtype):
    base = torch.randn(40, 300, device=DEV).to(dtype)
    for v in (base[:, 1:98], base[::3, 5:], base.t(), base[:, :64], base[:1].expand(9, 300), base.reshape(4, 10, 300)[:, 1:4],
              base[3:, ::2]):
        p, q = det.pack_int8(v), det.pack_int8(v.contiguous())
        assert torch.equal(p.codes, q.codes) and torch.equal(p.exponents, q.exponents)
        wide = torch.zeros(*v.shape[:-1], v.shape[-1] + 7, dtype=torch.int8, device=DEV)
        wide[..., 3:-4] = p.codes
        assert torch.equal(det.unpack_int8(det.PackedInt8(wide[..., 3:-4], p.exponents), dtype), det.unpack_int8(p, dtype))


def test_rows_past_32_bits():
    # 2^32 and more codes: one row of 2^24 + 8 would be refused, many rows are not
    N, C = 270000, 16384
    x = torch.zeros(N, C, dtype=BF16, device=DEV)
    x[-1] = torch.arange(C, device=DEV) % 120
    x[N // 2, 7] = -3.0
    p = det.pack_int8(x)
    y = det.unpack_int8(p, BF16)
    assert torch.equal(y, x)
    del y
    part = det.pack_int8(x[-2:])
    assert torch.equal(p.codes[-2:], part.codes) and torch.equal(p.exponents[-2:], part.exponents)


def test_graph_replays():
    buf = torch.randn(50, 77, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = det.pack_int8(buf)
        y = det.unpack_int8(p, BF16)
    for _ in range(3):
        buf.copy_(torch.randn(50, 77, device=DEV) * 100)
        graph.replay()
        q = det.pack_int8(buf)
        torch.cuda.synchronize()
        assert torch.equal(p.codes, q.codes) and torch.equal(p.exponents, q.exponents)
        assert torch.equal(y, det.unpack_int8(q, BF16))


@pytest.mark.parametrize("dtype,bias,N,C,F", [(BF16, False, 70, 96, 40), (F32, True, 33, 45, 20), (BF16, True, 300, 513, 64),
                                              (F32, False, 1, 1, 1)])
def test_det_linear_reads_its_input_back(dtype, bias, N, C, F):
    announce(f"DetLinear int8 {dtype} {bias} {N} {C} {F}")
    torch.manual_seed(2)
    plain = det.DetLinear(C, F, bias=bias, device=DEV, dtype=dtype)
    kept = det.DetLinear(C, F, bias=bias, device=DEV, dtype=dtype, checkpoint="int8")
    kept.load_state_dict(plain.state_dict())
    assert "int8" in repr(kept)
    x = torch.randn(2, N, C, device=DEV).to(dtype).requires_grad_(True)
    # the same results but for dW, which is that of the values read back
    y, z = plain(x), kept(x)
    assert torch.equal(y, z)
    gy = torch.randn_like(y)
    a, b = (torch.autograd.grad(t, [x, *m.parameters()], gy) for t, m in ((y, plain), (z, kept)))
    assert torch.equal(a[0], b[0]) and (not bias or torch.equal(a[2], b[2]))
    back = det.unpack_int8(det.pack_int8(x), dtype).requires_grad_(True)
    assert torch.equal(torch.autograd.grad(plain(back), plain.weight, gy)[0], b[1])
    # half a unit of the largest in a block: 1/127 of it
    assert ((back - x).abs() <= x.abs().amax(-1, keepdim=True) / 127).all()
    sizes = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append((t.dtype, t.numel())), t)[1], lambda t: t):
        kept(x)
    assert sorted(n for d, n in sizes if d == torch.int8) == sorted([2 * N * C, 2 * N * ((C + 31) // 32)])
    assert sum(n for d, n in sizes if d != torch.int8) == F * C
    # frozen weights: nothing of x is kept
    kept.requires_grad_(False)
    sizes.clear()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append(t.dtype), t)[1], lambda t: t):
        w = kept(x)
    assert torch.int8 not in sizes and torch.equal(torch.autograd.grad(w, x, gy)[0], a[0])
