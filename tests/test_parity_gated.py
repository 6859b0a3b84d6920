"""GPU parity: the gated block on codes, the gate by itself and its way back
against exact integer sums and 64-bit definitions."""
import pytest
import torch

import gated_util as gu
import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
ACTS = gu.ACTS


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def check(tq, M, F, K, ft, act, biases=(True, True), seed=0, lo=-127):
    dt = ref.TORCH[ft]
    qx, sx, qg, sg, qu, su, bg, bu = gu.operands(M, F, K, seed + M + F + K, dt, lo)
    bg, bu = (b if want else None for b, want in zip((bg, bu), biases))
    dev = [None if t is None else t.cuda() for t in (qx, sx, qg, sg, qu, su, bg, bu)]
    y, z = tq.tq_w8a8_gated_linear(*dev[:6], bias_gate=dev[6], bias_up=dev[7], act=act, out_dtype=dt, preact=True)
    assert y.shape == (M, F) and z.shape == (M, 2 * F) and y.dtype == z.dtype == dt
    (g, tg), (u, tu) = gu.project(qx, sx, qg, sg, bg), gu.project(qx, sx, qu, su, bu)
    wy, ty = gu.gate(g, tg, u, tu, act)
    ref.assert_within(z, torch.cat([g, u], 1), torch.cat([tg + ref.rounding(g, ft), tu + ref.rounding(u, ft)], 1), "z")
    ref.assert_within(y, wy, ty + ref.rounding(wy, ft), "y")
    alone = tq.tq_w8a8_gated_linear(*dev[:6], bias_gate=dev[6], bias_up=dev[7], act=act, out_dtype=dt)
    assert torch.equal(alone, y), "y changes with preact"
    return dev, y, z


# one token to several tiles; widths and depths off every tile, block and vector
@pytest.mark.parametrize("M,F,K", [(1, 1, 1), (1, 16, 64), (1, 65, 4096), (3, 17, 15), (5, 33, 100), (16, 128, 1000),
                                   (17, 36, 128), (33, 40, 272), (64, 127, 2064), (65, 65, 129), (100, 100, 2000),
                                   (128, 64, 128), (129, 129, 640), (200, 1, 96), (255, 256, 144), (256, 128, 256),
                                   (257, 192, 1008), (300, 130, 4097), (513, 257, 528), (2, 1500, 16), (70, 8, 17)])
@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_sizes(tq, M, F, K, ft):
    note("gated", M, F, K, ft)
    check(tq, M, F, K, ft, "silu")


# every tile size, with tiles that stick out on both sides and a K that ends inside a block
@pytest.mark.parametrize("M,F,K", [(1000, 550, 272), (1500, 800, 528), (2100, 1100, 144), (4100, 2055, 400),
                                   (2048, 4096, 1024), (40, 3100, 1040), (30, 3500, 208), (64, 2000, 1040),
                                   (250, 500, 400), (1201, 70, 1552), (220, 253, 2064), (40, 501, 1168)])
@pytest.mark.parametrize("ft,act", [("bf16", "gelu_tanh"), ("f32", "none"), ("f16", "relu")])
def test_tiles(tq, M, F, K, ft, act):
    note("gated tiles", M, F, K, ft)
    check(tq, M, F, K, ft, act)


# operands of other alignments: every number of whole blocks in flight, every tile size
@pytest.mark.parametrize("M,F,K", [(100, 65, k) for k in (1, 127, 129, 250, 257, 385, 513, 645, 1030)] +
                         [(1500, 800, 389), (1500, 803, 650), (2900, 2055, 131), (2900, 2055, 520), (4100, 2050, 261)])
def test_any_alignment(tq, M, F, K):
    note("gated any alignment", M, F, K)
    check(tq, M, F, K, "bf16", "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("biases", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("M,ft", [(4, "f16"), (90, "bf16"), (260, "f32")])
def test_activations_and_biases(tq, act, biases, M, ft):
    note("gated", act, biases, M, ft)
    check(tq, M, 132, 384, ft, act, biases)


@pytest.mark.parametrize("M", [1, 40, 130, 300])
def test_code_minus_128(tq, M):
    check(tq, M, 24, 2048, "f32", "relu", lo=-128)


@pytest.mark.parametrize("M", [5, 30, 70, 300])
def test_operands_that_start_anywhere(tq, M):
    F, K = 100, 512
    dev = [t.cuda() for t in gu.operands(M, F, K, M, torch.float32)]
    want = tq.tq_w8a8_gated_linear(*dev[:6], out_dtype=torch.float32)

    def moved(t, by):
        return torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")[by:].view(t.shape).copy_(t)
    for x, g, u in ((3, 0, 0), (0, 5, 0), (0, 0, 9), (1, 2, 4)):
        got = tq.tq_w8a8_gated_linear(moved(dev[0], x), dev[1], moved(dev[2], g), dev[3], moved(dev[4], u), dev[5],
                                      out_dtype=torch.float32)
        assert torch.equal(got, want), (x, g, u)


@pytest.mark.parametrize("M,F,K", [(1, 40, 512), (20, 72, 640), (100, 96, 384), (300, 200, 1040), (600, 700, 144)])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_kept_values_are_the_products(tq, M, F, K, ft):
    """z's bits are those of the two W8A8 products, and the gate of a stored z in
    binary32 has the block's bits."""
    dev, y, z = check(tq, M, F, K, ft, "silu")
    for j in range(2):
        alone = tq.tq_w8a8_linear_epilogue(dev[0], dev[1], dev[2 + 2 * j], dev[3 + 2 * j], bias=dev[6 + j],
                                           out_dtype=ref.TORCH[ft])
        assert torch.equal(z[:, j * F:(j + 1) * F], alone)
    if ft == "f32":
        assert torch.equal(tq.tq_gated_act(z, "silu"), y)


def test_a_token_alone_has_the_bits_it_has_in_a_batch(tq):
    dev = [t.cuda() for t in gu.operands(300, 100, 640, 2, torch.bfloat16)]
    full = tq.tq_w8a8_gated_linear(*dev[:6], bias_gate=dev[6], bias_up=dev[7])
    for m in (1, 20, 64, 65, 129, 256):
        part = tq.tq_w8a8_gated_linear(dev[0][:m], dev[1][:m], *dev[2:6], bias_gate=dev[6], bias_up=dev[7])
        assert torch.equal(part, full[:m]), m


def pair(M, F, ft, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, F), generator=g).to(ref.TORCH[ft]), (2 * torch.randn((M, 2 * F), generator=g)).to(ref.TORCH[ft]))


SHAPES = [(1, 1), (1, 8), (3, 5), (7, 7), (16, 512), (17, 513), (100, 519), (64, 520), (65, 9), (1000, 264), (4099, 24),
          (33, 1500), (5000, 3), (2, 11008), (1, 2)]
KINDS = [("none", "bf16"), ("relu", "f16"), ("silu", "f32"), ("silu", "bf16"), ("gelu", "bf16"), ("gelu", "f32"),
         ("gelu_tanh", "f32"), ("gelu_tanh", "f16")]


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("act,ft", KINDS)
def test_gate(tq, M, F, act, ft):
    note("gate", M, F, act, ft)
    _, z = pair(M, F, ft, M + F)
    g, u = z[:, :F].double(), z[:, F:].double()
    want, tol = gu.gate(g, 0 * g, u, 0 * u, act)
    ref.assert_within(tq.tq_gated_act(z.cuda(), act), want, tol + ref.rounding(want, ft), "y")


@pytest.mark.parametrize("M,F", SHAPES)
@pytest.mark.parametrize("act,ft", KINDS)
def test_gate_backward(tq, M, F, act, ft):
    note("gate backward", M, F, act, ft)
    dy, z = pair(M, F, ft, 3 * M + F)
    dz, db = tq.tq_gated_act_backward(dy.cuda(), z.cuda(), act)
    assert dz.shape == z.shape and dz.dtype == z.dtype and db.shape == (2 * F,) and db.dtype == torch.float32
    want, tol, raw = gu.gate_backward(dy, z, act, ft)
    ref.assert_within(dz, want, tol, "dz")
    # a column's terms go through at most M / 64 additions in a wave's rows and 64 beyond
    ref.assert_within(db, want.sum(0), (raw + (M / 64 + 64) * ref.U * want.abs()).sum(0) + 1e-30, "dbias")
    again = tq.tq_gated_act_backward(dy.cuda(), z.cuda(), act)
    assert torch.equal(again[0], dz) and torch.equal(again[1], db)


@pytest.mark.parametrize("act", ACTS)
def test_gate_backward_against_differences(tq, act):
    """dz against central differences of the gate's definition (step 1e-4 in 64
    bits: truncation below 1e-8 times |u|)."""
    z = torch.linspace(-6, 6, 514)[None].contiguous()
    if act == "relu":
        z = z + 0.011                                   # no difference across the corner
    F, h = 257, 1e-4
    dz, _ = tq.tq_gated_act_backward(torch.ones((1, F)).cuda(), z.cuda(), act)
    g, u = z[:, :F].double(), z[:, F:].double()

    def y(g, u):
        return ref.act(g, act) * u
    num = torch.cat([(y(g + h, u) - y(g - h, u)) / (2 * h), (y(g, u + h) - y(g, u - h)) / (2 * h)], 1)
    assert float((dz.cpu().double() - num).abs().max()) < 6 * (1e-8 + 32 * ref.U * 8)


@pytest.mark.parametrize("M", [1, 3, 64, 65, 300])
@pytest.mark.parametrize("F", [5, 8, 13, 512, 513, 519, 1030])
@pytest.mark.parametrize("act,ft", [("relu", "f32"), ("silu", "bf16"), ("gelu_tanh", "f16")])
def test_dz_over_z(tq, M, F, act, ft):
    note("gate backward in place", M, F, act, ft)
    dy, z = (t.cuda() for t in pair(M, F, ft, M * F))
    want, want_db = tq.tq_gated_act_backward(dy, z, act)
    n = tq.tq_gated_act_backward_workspace_bytes(M, F)
    db, ws = torch.empty(2 * F, device="cuda"), torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    s = tq._lib.tq_gated_act_backward(dy.data_ptr(), z.data_ptr(), tq.FTYPE[z.dtype], M, F, tq.ACT[act], z.data_ptr(),
                                      db.data_ptr(), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert s == 0 and torch.equal(z, want) and torch.equal(db, want_db)


@pytest.mark.parametrize("M,F", [(64, 513), (65, 7), (65, 519), (100, 50), (8192, 520), (8192, 5), (8193, 1001)])
def test_gate_backward_keeps_inside(tq, M, F):
    note("gate backward, guarded workspace", M, F)
    dy, z = (t.cuda() for t in pair(M, F, "f32", F))
    want = tq.tq_gated_act_backward(dy, z, "silu")
    n, G = tq.tq_gated_act_backward_workspace_bytes(M, F), 4096
    ws, bias = (torch.full((G + b + G,), 255, dtype=torch.uint8, device="cuda") for b in (n, 8 * F))
    dz = torch.empty_like(z)
    assert 0 == tq._lib.tq_gated_act_backward(dy.data_ptr(), z.data_ptr(), 0, M, F, tq.ACT["silu"], dz.data_ptr(),
                                              bias.data_ptr() + G, ws.data_ptr() + G if n else None, n,
                                              torch.cuda.current_stream().cuda_stream)
    for b, size in ((ws, n), (bias, 8 * F)):
        assert bool((b[:G] == 255).all()) and bool((b[G + size:] == 255).all())
    assert torch.equal(dz, want[0]) and torch.equal(bias[G:G + 8 * F].view(torch.float32), want[1])


@pytest.mark.parametrize("act", ACTS)
def test_extreme_values(tq, act):
    """Gates whose exponentials or cubes overflow binary32 on the way, infinities
    and NaN."""
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 100.0, -100.0, 1e13, -1e13, 1e20, -1e20, 3e38, -3e38,
                      0.7, -0.7])
    z = torch.cat([g, torch.full((16,), 0.5)])[None]
    y = tq.tq_gated_act(z.cuda(), act)
    a = ref.act(g.double(), act)
    ref.assert_within(y[0], 0.5 * a, 32 * ref.U * g.double().abs() * (a != 0) + 1e-37, "y")
    dz, db = tq.tq_gated_act_backward(torch.ones((1, 16)).cuda(), z.cuda(), act)
    slope = ref.act_slope(g.double(), act).nan_to_num(0.0)
    slope = torch.where(g.double().abs() > 50, (g > 0).double() if act != "none" else 1 + 0 * slope, slope)
    want = torch.cat([0.5 * slope, a])
    tol = torch.cat([32 * ref.U + 0 * slope, 32 * ref.U * g.double().abs() * (a != 0)])
    ref.assert_within(dz[0], want, tol + 1e-37, "dz")
    assert torch.equal(dz[0], db)
    # gates NaN, 1, inf, 2, 1 with the factors NaN, 1, inf, 3, 3
    odd = torch.tensor([[float("nan"), 1.0, float("inf"), 2.0, 1.0, float("nan"), 1.0, float("inf"), 3.0, 3.0]])
    y = tq.tq_gated_act(odd.cuda(), act).cpu()[0]
    assert torch.isnan(y[0]) and y[2] == float("inf") and torch.isfinite(y[[1, 3, 4]]).all()
    dz, _ = tq.tq_gated_act_backward(torch.ones((1, 5)).cuda(), odd.cuda(), act)
    dz = dz.cpu()[0]
    assert torch.isnan(dz[[0, 5]]).all() and dz[7] == float("inf") and torch.isfinite(dz[[1, 3, 4, 6, 8, 9]]).all()


def test_slope_zero_is_gradient_zero(tq):
    """relu's gate at or below 0 takes no gradient, whatever dy and u hold."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[-1.0, 0.0, -2.0, -1.0, 1.0, 1.0, inf, nan, 1.0, 1.0]])
    dz, _ = tq.tq_gated_act_backward(torch.tensor([[nan, 1.0, 1.0, inf, 2.0]]).cuda(), z.cuda(), "relu")
    assert dz.cpu()[0, :5].tolist() == [0.0, 0.0, 0.0, 0.0, 2.0]


def test_empty_and_refusals(tq):
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    f = lambda *s: torch.ones(s, device="cuda")
    call = tq.tq_w8a8_gated_linear
    y = call(i8(3, 0), f(3), i8(5, 0), f(5), i8(5, 0), f(5), bias_gate=2 * f(5), bias_up=3 * f(5), act="relu",
             out_dtype=torch.float32)
    assert torch.equal(y, 6 * f(3, 5))                  # empty sums: the biases alone
    assert call(i8(0, 8), f(0), i8(5, 8), f(5), i8(5, 8), f(5)).shape == (0, 5)
    assert call(i8(4, 8), f(4), i8(0, 8), f(0), i8(0, 8), f(0)).shape == (4, 0)
    dz, db = tq.tq_gated_act_backward(f(0, 9), f(0, 18), "silu")
    assert dz.shape == (0, 18) and db.shape == (18,) and not db.any()
    assert tq.tq_gated_act(f(0, 8)).shape == (0, 4) and tq.tq_gated_act(f(3, 0)).shape == (3, 0)
    good = (i8(3, 8), f(3), i8(5, 8), f(5), i8(5, 8), f(5))
    for at, bad, err in ((0, f(3, 8), TypeError), (2, i8(5, 9), ValueError), (4, i8(6, 8), ValueError),
                         (1, f(4), ValueError), (3, f(6), ValueError), (5, f(4), ValueError)):
        with pytest.raises(err):
            call(*good[:at], bad, *good[at + 1:])
    for more in ({"bias_gate": f(4)}, {"bias_up": f(6)}, {"bias_gate": f(5), "bias_up": f(5).half()}):
        with pytest.raises(ValueError):
            call(*good, **more)
    with pytest.raises(KeyError):
        call(*good, act="tanh")
    for bad in (f(3, 5), f(6)):
        with pytest.raises(ValueError):
            tq.tq_gated_act(bad)
    with pytest.raises(ValueError):
        tq.tq_gated_act_backward(f(3, 5), f(3, 8))
    with pytest.raises(ValueError):
        tq.tq_gated_act_backward(f(3, 4).half(), f(3, 8))
    with pytest.raises(tq.TQError):
        call(i8(1, 131072), f(1), i8(1, 131072), f(1), i8(1, 131072), f(1))    # sums would pass 32 bits
