"""GPU parity: the W8A8 product beside adapters of many requests against exact
integer sums and a 64-bit definition, adapter by adapter."""
import math

import pytest
import torch

import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
U = ref.U


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def operands(M, N, K, R, count, seed, ft, out):
    """A token's codes are independent of its x here: the two terms are checked apart."""
    g = torch.Generator().manual_seed(seed)
    qx, qw = (torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int64).to(torch.int8) for n in (M, N))
    sx = (0.5 + torch.rand(M, generator=g)) / 64
    sw = (0.5 + torch.rand(N, generator=g)) / (74 * max(1, K) ** 0.5)
    x = torch.randn((M, K), generator=g).to(ref.TORCH[ft])
    a = (torch.randn((count, R, K), generator=g) / max(1, K) ** 0.5).to(ref.TORCH[ft])
    b = (torch.randn((count, N, R), generator=g) / R ** 0.5).to(ref.TORCH[ft])
    scale = 0.5 + torch.rand(count, generator=g)
    adapter = torch.randint(-1, count, (M,), generator=g, dtype=torch.int32)
    bias = torch.randn(N, generator=g).to(ref.TORCH[out])
    res = torch.randn((M, N), generator=g).to(ref.TORCH[out])
    return x, qx, sx, qw, sw, adapter, a, b, scale, bias, res


def definition(x, qx, sx, qw, sw, adapter, a, b, scale, bias, res, act, ft, out):
    """(z, y, their bounds).  h is off by its sum's depth (K / 64 products in a lane
    of the longest form, 80 joins) and two roundings; in the product it holds 16 bits
    or 22 (f16), and the sum over the ranks goes through R + 8 additions."""
    M, N, K, R = qx.shape[0], qw.shape[0], qx.shape[1], a.shape[1]
    acc = qx.double() @ qw.double().t() if K else torch.zeros(M, N, dtype=torch.float64)
    z = acc * sx.double()[:, None] * sw.double()
    low, t_low = torch.zeros_like(z), torch.zeros_like(z)
    split = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16}[ft]
    for c in range(a.shape[0]):
        rows = adapter == c
        f = 1.0 if scale is None else scale[c].double()
        h = f * (x[rows].double() @ a[c].double().t())
        mag = f * (x[rows].double().abs() @ a[c].double().abs().t())
        low[rows] = h @ b[c].double().t()
        # f16 pieces are relative to the row's largest h
        top = h.abs().amax(1, keepdim=True).expand_as(h) if ft == "f16" else h.abs()
        th = (K / 64 + 84) * U * mag + split * (top + h.abs())
        t_low[rows] = (th + (R + 8) * U * h.abs()) @ b[c].double().abs().t()
    tz = 4 * U * (z.abs() + low.abs() + (0 if bias is None else bias.double().abs())) + t_low
    z = z + low + (0 if bias is None else bias.double())
    y = ref.act(z, act)
    ty = 1.2 * tz + (0 if act in ("none", "relu") else 24 * U * z.abs())
    if res is not None:
        y = y + res.double()
        ty = ty + U * (y.abs() + res.double().abs())
    return z, y, tz + ref.rounding(z, out), ty + ref.rounding(y, out)


def check(tq, M, N, K, R, count, ft, out=None, act="silu", seed=0, sort=False, parts=(True, True, True), adapter=None):
    out = out or ft
    ops = list(operands(M, N, K, R, count, seed + M + N + K + R, ft, out))
    if sort:
        ops[5] = ops[5].sort().values
    if adapter is not None:
        ops[5] = adapter
    for at, keep in zip((8, 9, 10), parts):
        if not keep:
            ops[at] = None
    dev = [None if t is None else t.cuda() for t in ops]
    y, z = tq.tq_w8a8_linear_adapters(*dev[:8], scale=dev[8], bias=dev[9], act=act, residual=dev[10],
                                      out_dtype=ref.TORCH[out], preact=True)
    wz, wy, tz, ty = definition(*ops, act, ft, out)
    ref.assert_within(z, wz, tz, "z")
    ref.assert_within(y, wy, ty, "y")
    alone = tq.tq_w8a8_linear_adapters(*dev[:8], scale=dev[8], bias=dev[9], act=act, residual=dev[10],
                                       out_dtype=ref.TORCH[out])
    assert torch.equal(alone, y), "y changes with preact"
    # a token without an adapter has the plain product's bits
    none = (ops[5] < 0) | (ops[5] >= count)
    if bool(none.any()):
        plain = tq.tq_w8a8_linear_epilogue(*dev[1:5], bias=dev[9], act=act, residual=dev[10], out_dtype=ref.TORCH[out])
        assert torch.equal(y.cpu()[none], plain.cpu()[none]), "a token without an adapter"
    return dev, y


# one token to several tiles; widths, depths and ranks off every tile, block and vector
@pytest.mark.parametrize("M,N,K,R,count", [(1, 1, 1, 1, 1), (1, 16, 64, 8, 3), (1, 130, 4096, 16, 8), (3, 17, 15, 3, 2),
                                           (5, 33, 100, 5, 9), (16, 256, 1000, 16, 4), (17, 72, 128, 32, 20),
                                           (33, 40, 272, 64, 7), (64, 127, 2064, 12, 70), (65, 129, 129, 33, 2),
                                           (100, 200, 2000, 16, 5), (128, 128, 128, 100, 3), (129, 257, 640, 8, 50),
                                           (200, 1, 96, 1, 4), (255, 512, 144, 15, 3), (257, 384, 1008, 40, 6),
                                           (300, 260, 4097, 17, 8), (513, 515, 528, 64, 11), (2, 3000, 16, 24, 2),
                                           (70, 8, 17, 200, 3), (48, 640, 1040, 256, 6)])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_sizes(tq, M, N, K, R, count, ft):
    note("adapters", M, N, K, R, count, ft)
    check(tq, M, N, K, R, count, ft)


# every tile size, tokens in the order of their requests and in any
@pytest.mark.parametrize("M,N,K,R", [(1000, 1100, 272, 16), (1500, 1600, 528, 64), (2100, 2200, 144, 7),
                                     (4100, 4110, 400, 16), (40, 6200, 1040, 8), (30, 7000, 208, 32),
                                     (64, 4000, 1040, 16), (250, 1000, 400, 48), (1201, 140, 1552, 16),
                                     (220, 507, 2064, 9), (40, 1001, 1168, 16)])
@pytest.mark.parametrize("ft,out,sort", [("bf16", "bf16", True), ("f16", "f32", False), ("f32", "f16", True)])
def test_tiles(tq, M, N, K, R, ft, out, sort):
    note("adapters tiles", M, N, K, R, ft, out, sort)
    check(tq, M, N, K, R, 5, ft, out, act="none" if sort else "gelu_tanh", sort=sort)


# either side of the rules of the few-token kernel, adapters in any order
@pytest.mark.parametrize("M,N,K,R", [(90, 4300, 272, 16), (128, 4096, 144, 64), (130, 3270, 208, 63), (128, 4097, 144, 64),
                                     (32, 6145, 135, 9), (33, 8192, 129, 8), (33, 8193, 144, 8),
                                     (200, 4096, 144, 64), (256, 1000, 135, 64), (257, 1000, 144, 64)])
@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_few_token_rules(tq, M, N, K, R, ft):
    note("adapters rules", M, N, K, R, ft)
    check(tq, M, N, K, R, 90, ft)


# codes whose rows start anywhere: every tile of that kernel
@pytest.mark.parametrize("M,N,K", [(100, 130, 127), (100, 130, 513), (530, 540, 259), (1500, 1600, 389),
                                   (2900, 4110, 131)])
@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_any_alignment(tq, M, N, K, ft):
    note("adapters any alignment", M, N, K, ft)
    check(tq, M, N, K, 16, 4, ft, sort=True)


@pytest.mark.parametrize("parts", [(False, False, False), (True, False, True), (False, True, False)])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N", [(6, 264), (150, 264), (600, 568)])
def test_parts(tq, parts, act, M, N):
    check(tq, M, N, 384, 16, 3, "bf16", act=act, parts=parts)


@pytest.mark.parametrize("M", [3, 40, 200, 600])
def test_ids_outside_are_none(tq, M):
    """Every value that is no adapter, and batches where nobody has one."""
    ids = torch.tensor([-1, 3, 2, -2 ** 31, 0, 2 ** 31 - 1, 1, 4])[torch.arange(M) % 8].int()
    N = 200 if M < 600 else 520
    check(tq, M, N, 256, 16, 3, "bf16", adapter=ids)
    check(tq, M, N, 256, 16, 3, "f16", adapter=torch.full((M,), -1, dtype=torch.int32))


@pytest.mark.parametrize("M", [1, 12, 40, 130, 300, 700])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_other_adapters_do_not_reach_a_token(tq, M, ft):
    """Infinities and NaN in adapters, their scales and their tokens stay with them."""
    N, K, R, count = 300 if M < 700 else 900, 272, 16, 6
    ops = [t.cuda() for t in operands(M, N, K, R, count, M, ft, "f32")]
    want = tq.tq_w8a8_linear_adapters(*ops[:8], scale=ops[8], out_dtype=torch.float32)
    bad = [t.clone() for t in ops]
    bad[6][1, 3, 5], bad[7][2, 7] = float("nan"), float("inf")
    bad[8][4] = float("nan")
    gone = ops[5] == 3
    bad[0][gone] = float("inf")
    got = tq.tq_w8a8_linear_adapters(*bad[:8], scale=bad[8], out_dtype=torch.float32)
    keep = (ops[5] != 1) & (ops[5] != 2) & (ops[5] != 4) & ~gone
    assert torch.equal(got[keep], want[keep])
    spoilt = (ops[5] == 1) | (ops[5] == 4)
    assert bool(torch.isnan(got[spoilt]).all())
    assert not bool(torch.isfinite(got[gone]).any())
    two = ops[5] == 2                                   # one row of b is infinite: that column alone
    col = torch.arange(N, device="cuda") == 7
    assert torch.equal(got[two][:, ~col], want[two][:, ~col]) and not bool(torch.isfinite(got[two][:, col]).any())


@pytest.mark.parametrize("M", [4, 200, 600])
@pytest.mark.parametrize("ft,size", [("f16", 1e-7), ("f16", 300.0), ("bf16", 1e30), ("bf16", 1e-25), ("f32", 1e25)])
def test_low_values_far_from_one(tq, M, ft, size):
    """h beyond f16's range on either side, and near the ends of binary32's."""
    N, K, R, count = 130 if M < 600 else 500, 256, 16, 3
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g).to(ref.TORCH[ft])
    a = (torch.randn((count, R, K), generator=g) * (size if ft != "f16" else min(size, 300.0))).to(ref.TORCH[ft])
    b = torch.randn((count, N, R), generator=g).to(ref.TORCH[ft])
    scale = torch.full((count,), 50.0 if ft == "f16" and size > 1 else 1.0)
    adapter = torch.arange(M, dtype=torch.int32) % count
    zero = torch.zeros((M, K), dtype=torch.int8), torch.ones(M), torch.zeros((N, K), dtype=torch.int8), torch.ones(N)
    ops = (x, *zero, adapter, a, b, scale, None, None)
    y = tq.tq_w8a8_linear_adapters(*(t.cuda() for t in ops[:8]), scale=scale.cuda(), out_dtype=torch.float32)
    _, want, _, tol = definition(*ops, "none", ft, "f32")
    ref.assert_within(y, want, tol, "y")


def test_strides_and_odd_addresses(tq):
    for M in (5, 70, 300, 600):
        N, K, R, count = 136 if M < 600 else 520, 272, 13, 4
        ops = [t.cuda() for t in operands(M, N, K, R, count, 8, "bf16", "bf16")]
        want = tq.tq_w8a8_linear_adapters(*ops[:8], scale=ops[8], bias=ops[9], residual=ops[10])

        def inside(t):
            wide = torch.full((M, t.shape[1] + 7), float("nan"), dtype=t.dtype, device="cuda")
            wide[:, 3:3 + t.shape[1]] = t
            return wide[:, 3:3 + t.shape[1]]

        def moved(t, by):
            return torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")[by:].view(t.shape).copy_(t)
        got = tq.tq_w8a8_linear_adapters(inside(ops[0]), *ops[1:6], moved(ops[6], 1), moved(ops[7], 3), scale=ops[8],
                                         bias=ops[9], residual=inside(ops[10]))
        assert torch.equal(got, want), M


@pytest.mark.parametrize("M,R", [(1, 16), (40, 9), (300, 33), (700, 64)])
def test_keeps_inside_its_workspace(tq, M, R):
    N, K, count, G = 200 if M < 700 else 520, 272, 3, 4096
    ops = [t.cuda() for t in operands(M, N, K, R, count, 9, "bf16", "bf16")]
    want = tq.tq_w8a8_linear_adapters(*ops[:8], scale=ops[8])
    n = tq.tq_w8a8_linear_adapters_workspace_bytes(M, R)
    assert n >= M * R * 4
    ws, out = (torch.full((G + size + G,), 255, dtype=torch.uint8, device="cuda") for size in (n, 2 * M * N))
    x, qx, sx, qw, sw, ids, a, b, scale = (t.data_ptr() for t in ops[:9])
    assert 0 == tq._lib.tq_w8a8_linear_adapters(x, 2, K, qx, sx, qw, sw, M, N, K, ids, count, R, a, b, scale, None, 0, 0,
                                                None, N, out.data_ptr() + G, None, 2, ws.data_ptr() + G, n,
                                                torch.cuda.current_stream().cuda_stream)
    for t, size in ((ws, n), (out, 2 * M * N)):
        assert bool((t[:G] == 255).all()) and bool((t[G + size:] == 255).all())
    assert torch.equal(out[G:G + 2 * M * N].view(torch.bfloat16).view(M, N), want)


def test_empty_and_refusals(tq):
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")
    ids = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    call = tq.tq_w8a8_linear_adapters
    good = (f(3, 8), i8(3, 8), f(3), i8(5, 8), f(5), ids(3), f(2, 4, 8), f(2, 5, 4))
    assert torch.equal(call(*good, out_dtype=torch.float32), 32 * f(3, 5))
    # no adapters at all, no K, no tokens, no columns
    y = call(*good[:6], f(0, 4, 8), f(0, 5, 4), bias=2 * f(5), out_dtype=torch.float32)
    assert torch.equal(y, 2 * f(3, 5))
    y = call(f(3, 0), i8(3, 0), f(3), i8(5, 0), f(5), ids(3), f(2, 4, 0), f(2, 5, 4), bias=2 * f(5),
             out_dtype=torch.float32)
    assert torch.equal(y, 2 * f(3, 5))
    assert call(f(0, 8), i8(0, 8), f(0), i8(5, 8), f(5), ids(0), f(2, 4, 8), f(2, 5, 4)).shape == (0, 5)
    assert call(f(3, 8), i8(3, 8), f(3), i8(0, 8), f(0), ids(3), f(2, 4, 8), f(2, 0, 4)).shape == (3, 0)
    for at, bad, err in ((0, f(3, 9), ValueError), (0, f(3, 8).half(), ValueError), (1, f(3, 8), TypeError),
                         (2, f(4), ValueError), (3, i8(5, 9), ValueError), (5, ids(4), ValueError),
                         (5, ids(3).long(), ValueError), (6, f(2, 4, 9), ValueError), (6, f(2, 3, 8), ValueError),
                         (7, f(1, 5, 4), ValueError), (7, f(2, 5, 4).half(), ValueError)):
        with pytest.raises(err):
            call(*good[:at], bad, *good[at + 1:])
    for more in ({"scale": f(3)}, {"bias": f(4)}, {"residual": f(3, 5)}):     # not the output's type
        with pytest.raises(ValueError):
            call(*good, **more)
    with pytest.raises(tq.TQError):
        call(*good[:6], f(2, 257, 8), f(2, 5, 257))
    with pytest.raises(tq.TQError):
        call(*good[:6], f(2, 0, 8), f(2, 5, 0))
