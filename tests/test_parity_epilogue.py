"""GPU parity: the W8A8 product with bias, activation and residual, and the
backward of that epilogue, against exact integer sums and 64-bit definitions."""
import pytest
import torch

import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def operands(M, N, K, seed, ft="bf16", full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    qx = torch.randint(lo, 128, (M, K), generator=g, dtype=torch.int64).to(torch.int8)
    qw = torch.randint(lo, 128, (N, K), generator=g, dtype=torch.int64).to(torch.int8)
    sx = (0.5 + torch.rand(M, generator=g)) / 64
    sw = (0.5 + torch.rand(N, generator=g)) / (74 * max(1, K) ** 0.5)
    bias = torch.randn(N, generator=g).to(ref.TORCH[ft])
    res = torch.randn((M, N), generator=g).to(ref.TORCH[ft])
    return qx, sx, qw, sw, bias, res


def product(qx, qw):
    return (qx.double() @ qw.double().t()) if qx.shape[1] else torch.zeros(qx.shape[0], qw.shape[0], dtype=torch.float64)


def check(tq, M, N, K, ft, act, bias, residual, seed=0, full=False):
    qx, sx, qw, sw, b, r = operands(M, N, K, seed + M + N + K, ft, full)
    b, r = (b if bias else None), (r if residual else None)
    dev = [None if t is None else t.cuda() for t in (qx, sx, qw, sw, b, r)]
    y, z = tq.tq_w8a8_linear_epilogue(*dev[:4], bias=dev[4], act=act, residual=dev[5], out_dtype=ref.TORCH[ft],
                                      preact=True)
    acc = product(qx, qw)                              # below 2^53: exact
    wz, wy = ref.epilogue(acc, sx, sw, b, act, r)
    tz, ty = ref.epilogue_tol(acc, sx, sw, b, act, r, ft)
    ref.assert_within(z, wz, tz, "preact")
    ref.assert_within(y, wy, ty, "y")
    alone = tq.tq_w8a8_linear_epilogue(*dev[:4], bias=dev[4], act=act, residual=dev[5], out_dtype=ref.TORCH[ft])
    assert torch.equal(alone, y), "y changes with preact"


# one token to several tiles; widths and depths off every tile, block and vector
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 64), (1, 130, 4096), (3, 17, 15), (5, 33, 100), (16, 256, 1000),
                                   (17, 72, 128), (33, 40, 272), (64, 127, 2064), (65, 129, 129), (100, 200, 2000),
                                   (128, 128, 128), (129, 257, 640), (200, 1, 96), (255, 512, 144), (256, 256, 256),
                                   (257, 384, 1008), (300, 260, 4097), (513, 515, 528), (2, 3000, 16), (70, 8, 17)])
@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_sizes(tq, M, N, K, ft):
    note("product", M, N, K, ft)
    check(tq, M, N, K, ft, "gelu_tanh", True, True)


# every tile size, with tiles that stick out on both sides and a K that ends inside a block
@pytest.mark.parametrize("M,N,K", [(1000, 1100, 272), (1500, 1600, 528), (2100, 2200, 144), (4100, 4110, 400),
                                   (4096, 4096, 2048), (40, 6200, 1040), (30, 7000, 208), (64, 4000, 1040),
                                   (250, 1000, 400), (1201, 140, 1552), (220, 507, 2064), (40, 1001, 1168)])
@pytest.mark.parametrize("ft,act", [("bf16", "silu"), ("f32", "none")])
def test_tiles(tq, M, N, K, ft, act):
    note("product tiles", M, N, K, ft)
    check(tq, M, N, K, ft, act, True, ft == "bf16")


# operands of other alignments: every number of whole blocks in flight, every tile size
@pytest.mark.parametrize("M,N,K", [(100, 130, k) for k in (1, 127, 129, 250, 257, 385, 513, 645, 1030)] +
                         [(1500, 1600, 389), (1500, 1600, 650), (2900, 4110, 131), (2900, 4110, 520), (4100, 4100, 261)])
def test_any_alignment(tq, M, N, K):
    note("product any alignment", M, N, K)
    check(tq, M, N, K, "bf16", "silu", True, True)


@pytest.mark.parametrize("M", [5, 30, 70, 300])
def test_operands_that_start_anywhere(tq, M):
    N, K = 200, 512
    g = torch.Generator().manual_seed(M)
    qx = torch.randint(-128, 128, (M * K + 3,), generator=g, dtype=torch.int8)[3:].view(M, K)
    qw = torch.randint(-128, 128, (N * K + 9,), generator=g, dtype=torch.int8)[9:].view(N, K)
    dx, dw = (torch.empty(v.numel() + 5, dtype=torch.int8, device="cuda")[5:].view(v.shape).copy_(v) for v in (qx, qw))
    one = torch.ones
    y = tq.tq_w8a8_linear_epilogue(dx, one(M).cuda(), dw, one(N).cuda(), out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), qx.double() @ qw.double().T)    # sums below 2^24


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,ft", [(4, "f16"), (90, "bf16"), (260, "f32"), (260, "f16")])
def test_epilogues(tq, act, bias, residual, M, ft):
    note("epilogue", act, bias, residual, M, ft)
    check(tq, M, 264, 384, ft, act, bias, residual)


@pytest.mark.parametrize("M", [1, 40, 130, 300])
def test_code_minus_128_and_the_longest_sums(tq, M):
    check(tq, M, 48, 2048, "f32", "none", False, False, full=True)
    K = 131071
    qx = torch.full((M, K), -128, dtype=torch.int8)
    qw = torch.full((3, K), -128, dtype=torch.int8)
    qw[1] = 127
    one = torch.ones
    y = tq.tq_w8a8_linear_epilogue(qx.cuda(), one(M).cuda(), qw.cuda(), one(3).cuda(), out_dtype=torch.float32)
    want = torch.tensor([K * 16384, -K * 128 * 127, K * 16384], dtype=torch.float32)
    assert torch.equal(y.cpu(), want.expand(M, 3))


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (48, 384, 1024), (100, 256, 512), (130, 128, 256), (512, 640, 1152)])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_plain_product_has_the_linears_bits(tq, M, N, K, ft):
    qx, sx, qw, sw, _, _ = (t.cuda() for t in operands(M, N, K, 5))
    a = tq.tq_w8a8_linear(qx, sx, qw, sw, out_dtype=ref.TORCH[ft])
    b = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, out_dtype=ref.TORCH[ft])
    assert torch.equal(a, b)


@pytest.mark.parametrize("M", [2, 70, 300])
def test_strided_residual_and_odd_addresses(tq, M):
    N, K = 136, 272
    qx, sx, qw, sw, bias, res = (t.cuda() for t in operands(M, N, K, 8))
    wide = torch.randn((M, N + 7), device="cuda").to(torch.bfloat16)
    r = wide[:, 3:3 + N]
    y = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, bias=bias, act="silu", residual=r)
    y2 = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, bias=bias, act="silu", residual=r.contiguous())
    assert torch.equal(y, y2)
    # the codes one byte off every alignment
    flat = torch.zeros(M * K + 1, dtype=torch.int8, device="cuda")
    flat[1:] = qx.reshape(-1)
    wflat = torch.zeros(N * K + 3, dtype=torch.int8, device="cuda")
    wflat[3:] = qw.reshape(-1)
    y3 = tq.tq_w8a8_linear_epilogue(flat[1:].view(M, K), sx, wflat[3:].view(N, K), sw, bias=bias, act="silu",
                                    residual=r)
    assert torch.equal(y, y3)


def test_a_token_alone_has_the_bits_it_has_in_a_batch(tq):
    qx, sx, qw, sw, bias, res = (t.cuda() for t in operands(300, 200, 640, 2))
    full = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, bias=bias, act="gelu", residual=res)
    for m in (1, 20, 64, 65, 129, 256):
        part = tq.tq_w8a8_linear_epilogue(qx[:m], sx[:m], qw, sw, bias=bias, act="gelu", residual=res[:m])
        assert torch.equal(part, full[:m]), m


@pytest.mark.parametrize("act", ACTS)
def test_extreme_values(tq, act):
    """Values whose exponentials or cubes overflow binary32 on the way."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 100.0, -100.0, 1e13, -1e13, 1e20, -1e20, 3e38, -3e38,
                      0.7, -0.7])
    qx = torch.ones((1, 1), dtype=torch.int8)
    qw = torch.ones((16, 1), dtype=torch.int8)
    y = tq.tq_w8a8_linear_epilogue(qx.cuda(), torch.ones(1).cuda(), qw.cuda(), z.cuda(), act=act,
                                   out_dtype=torch.float32)
    want = ref.act(z.double()[None], act)
    ref.assert_within(y, want, 32 * ref.U * z.double().abs()[None] * (want != 0) + 1e-37, "y")
    one = torch.ones((1, 16))
    dz, db = tq.tq_linear_epilogue_backward(one.cuda(), z[None].cuda(), act)
    slope = ref.act_slope(z.double(), act).nan_to_num(0.0)
    slope = torch.where(z.double().abs() > 50, (z > 0).double() if act != "none" else one[0].double(), slope)
    ref.assert_within(dz[0], slope, 32 * ref.U * one[0].double() + 1e-37, "dz")
    assert torch.equal(dz[0], db)


@pytest.mark.parametrize("M,N", [(1, 1), (1, 8), (3, 5), (7, 7), (16, 512), (17, 513), (100, 519), (64, 520),
                                 (1000, 264), (4099, 24), (33, 1500), (5000, 3), (2, 11008)])
@pytest.mark.parametrize("act,ft", [("none", "bf16"), ("relu", "f16"), ("silu", "f32"), ("gelu", "bf16"),
                                    ("gelu_tanh", "f32"), ("gelu_tanh", "f16")])
def test_epilogue_backward(tq, M, N, act, ft):
    note("epilogue backward", M, N, act, ft)
    g = torch.Generator().manual_seed(M + N)
    dy, z = (torch.randn((M, N), generator=g).to(ref.TORCH[ft]) for _ in range(2))
    dz, db = tq.tq_linear_epilogue_backward(dy.cuda(), (2 * z).cuda(), act)
    want = dy.double() * ref.act_slope((2 * z).double(), act)
    tol = 32 * ref.U * dy.double().abs() * (1 + (2 * z).double().abs())
    ref.assert_within(dz, want, tol + ref.rounding(want, ft), "dz")
    R = M / 64 + 64
    ref.assert_within(db, want.sum(0), (tol + R * ref.U * want.abs()).sum(0) + 1e-30, "dbias")
    again = tq.tq_linear_epilogue_backward(dy.cuda(), (2 * z).cuda(), act)
    assert torch.equal(again[0], dz) and torch.equal(again[1], db)


@pytest.mark.parametrize("act", ACTS[2:])
def test_slope_against_differences(tq, act):
    """dz against central differences of the forward pass's own definition
    (step 1e-4 in 64 bits: truncation below 1e-8)."""
    z = torch.linspace(-6, 6, 512)[None]
    dz, _ = tq.tq_linear_epilogue_backward(torch.ones_like(z).cuda(), z.cuda(), act)
    h = 1e-4
    num = (ref.act(z.double() + h, act) - ref.act(z.double() - h, act)) / (2 * h)
    assert float((dz.cpu().double() - num).abs().max()) < 1e-8 + 32 * ref.U * 8


def test_empty_and_refusals(tq):
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")
    y = tq.tq_w8a8_linear_epilogue(i8(3, 0), f(3), i8(5, 0), f(5), bias=2 * f(5), act="relu", out_dtype=torch.float32)
    assert torch.equal(y, 2 * f(3, 5))                  # empty sums: the bias alone
    assert tq.tq_w8a8_linear_epilogue(i8(0, 8), f(0), i8(5, 8), f(5)).shape == (0, 5)
    dz, db = tq.tq_linear_epilogue_backward(f(0, 9), f(0, 9), "silu")
    assert dz.shape == (0, 9) and not db.any()
    with pytest.raises(TypeError):
        tq.tq_w8a8_linear_epilogue(f(3, 8), f(3), i8(5, 8), f(5))
    with pytest.raises(ValueError):
        tq.tq_w8a8_linear_epilogue(i8(3, 8), f(3), i8(5, 9), f(5))
    with pytest.raises(ValueError):
        tq.tq_w8a8_linear_epilogue(i8(3, 8), f(2), i8(5, 8), f(5))
    with pytest.raises(ValueError):
        tq.tq_w8a8_linear_epilogue(i8(3, 8), f(3), i8(5, 8), f(5), bias=f(4))
    with pytest.raises(ValueError):
        tq.tq_w8a8_linear_epilogue(i8(3, 8), f(3), i8(5, 8), f(5), residual=f(3, 5))   # not the output's type
    with pytest.raises(KeyError):
        tq.tq_w8a8_linear_epilogue(i8(3, 8), f(3), i8(5, 8), f(5), act="tanh")
    with pytest.raises(tq.TQError):
        tq.tq_w8a8_linear_epilogue(i8(1, 131072), f(1), i8(1, 131072), f(1))           # sums would pass 32 bits
    with pytest.raises(ValueError):
        tq.tq_linear_epilogue_backward(f(3, 4), f(3, 5))
