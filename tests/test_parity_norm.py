"""GPU parity: layer norm, its fused per-token quantizer and its backward
against 64-bit definitions, under bounds derived from the kernels' sums."""
import numpy as np
import pytest
import torch

import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def draw(shape, ft, seed, mean=0.5, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((shape[0], 1), generator=g)
    return ((torch.randn(shape, generator=g) * spread + mean * rows)).to(ref.TORCH[ft])


def params(cols, wt, seed):
    g = torch.Generator().manual_seed(seed + 1000)
    return ((1 + 0.2 * torch.randn(cols, generator=g)).to(ref.TORCH[wt]),
            (0.3 * torch.randn(cols, generator=g)).to(ref.TORCH[wt]))


# every variant's width, its neighbours, widths below one vector, past the held rows
WIDTHS = [1, 7, 8, 9, 64, 511, 512, 520, 1000, 1024, 1025, 2048, 2056, 4095, 4096, 4100, 8192, 8200, 16384, 16391]


@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward_and_backward(tq, ft, cols):
    forward_and_backward(tq, ft, 5 if cols > 1024 else 37, cols)


# rows of a few elements, and rows that no workgroup holds, over several chunks of rows
@pytest.mark.parametrize("ft", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(70000, 2), (700, 3), (257, 7), (1100, 8209), (1030, 16400), (70, 20001)])
def test_short_and_long_rows(tq, ft, rows, cols):
    forward_and_backward(tq, ft, rows, cols)


def forward_and_backward(tq, ft, rows, cols):
    wt = "f32" if cols % 2 else ft
    note("norm", ft, wt, rows, cols)
    x, dy = draw((rows, cols), ft, cols), draw((rows, cols), ft, cols + 1, mean=0.1)
    w, b = params(cols, wt, cols)
    y, mean, rstd = tq.tq_layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5)
    wy, wm, wr, _ = ref.layer_norm(x, w, b, 1e-5)
    ty, tm, tr = ref.layer_norm_tol(x, w, b, 1e-5, ft)
    ref.assert_within(y, wy, ty, "y")
    ref.assert_within(mean, wm[:, 0], tm[:, 0], "mean")
    ref.assert_within(rstd, wr[:, 0], tr[:, 0], "rstd")

    dx, dw, db = tq.tq_layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    m, r = mean.cpu(), rstd.cpu()
    want = ref.layer_norm_backward(dy, x, w, m, r)
    tol = ref.layer_norm_backward_tol(dy, x, w, m, r, ft, wt)
    for name, got, wv, tv in zip(("dx", "dw", "db"), (dx, dw, db), want, tol):
        ref.assert_within(got, wv, tv, name)
    assert dw.dtype == w.dtype and dx.dtype == x.dtype


@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 8), (2, 5), (33, 1000), (17, 2056), (4, 4095), (9, 8192),
                                       (2, 16384), (2, 20001), (600, 3), (300, 7)])
def test_fused_quantizer_is_the_two_calls(tq, ft, rows, cols):
    """Codes and scales are bit for bit those of the norm followed by the
    per-token quantizer, zero rows and rows of one value included."""
    note("norm+quantize", ft, rows, cols)
    x = draw((rows, cols), ft, 7 * cols + rows)
    x[0] = 3.0                                         # no spread: y is the bias
    w, b = params(cols, ft, cols)
    if rows > 1:
        b = torch.zeros_like(b)                        # then that row is all zeros: scale 1
    q, s, mean, rstd = tq.tq_layer_norm_quant_per_token(x.cuda(), w.cuda(), b.cuda(), 1e-5, stats=True)
    y, m2, r2 = tq.tq_layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5)
    q2, s2, _ = tq.tq_quant_per_token(y, "s8")
    assert torch.equal(q.view(torch.uint8), q2) and torch.equal(s, s2)
    assert torch.equal(mean, m2) and torch.equal(rstd, r2)
    q3, s3 = tq.tq_layer_norm_quant_per_token(x.cuda(), w.cuda(), b.cuda(), 1e-5)
    assert torch.equal(q, q3) and torch.equal(s, s3)


@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_without_parameters_and_many_rows(tq, ft):
    x, dy = draw((1500, 264), ft, 3), draw((1500, 264), ft, 4)
    y, mean, rstd = tq.tq_layer_norm(x.cuda(), eps=0.0)
    ref.assert_within(y, ref.layer_norm(x, None, None, 0.0)[0], ref.layer_norm_tol(x, None, None, 0.0, ft)[0], "y")
    dx, dw, db = tq.tq_layer_norm_backward(dy.cuda(), x.cuda(), None, mean, rstd)
    m, r = mean.cpu(), rstd.cpu()
    want = ref.layer_norm_backward(dy, x, None, m, r)
    tol = ref.layer_norm_backward_tol(dy, x, None, m, r, ft, "f32")
    for name, got, wv, tv in zip(("dx", "dw", "db"), (dx, dw, db), want, tol):
        ref.assert_within(got, wv, tv, name)
    again = tq.tq_layer_norm_backward(dy.cuda(), x.cuda(), None, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again)), "the sums' order changed"


@pytest.mark.parametrize("cols", [256, 1001, 9000])
def test_row_strides_and_odd_addresses(tq, cols):
    """Column slices of a wider matrix, starting at odd elements."""
    wide, dwide = draw((11, cols + 9), "bf16", 1).cuda(), draw((11, cols + 9), "bf16", 2).cuda()
    w, b = (p.cuda() for p in params(cols + 1, "bf16", 5))
    x, dy = wide[:, 3:3 + cols], dwide[:, 5:5 + cols]
    w, b = w[1:], b[1:]
    y, mean, rstd = tq.tq_layer_norm(x, w, b, 1e-5)
    y2, m2, r2 = tq.tq_layer_norm(x.contiguous(), w.clone(), b.clone(), 1e-5)
    assert torch.equal(y, y2) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    a = tq.tq_layer_norm_backward(dy, x, w, mean, rstd)
    c = tq.tq_layer_norm_backward(dy.contiguous(), x.contiguous(), w.clone(), mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    q, s = tq.tq_layer_norm_quant_per_token(x, w, b)
    q2, s2 = tq.tq_layer_norm_quant_per_token(x.contiguous(), w, b)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_large_mean_keeps_the_variance(tq):
    """A mean 1e4 times the spread: the variance is taken around it."""
    x = draw((4, 4096), "f32", 9, mean=0.0) + 1.0e4
    y, mean, rstd = tq.tq_layer_norm(x.cuda(), eps=0.0)
    wy, _, wr, _ = ref.layer_norm(x, None, None, 0.0)
    ref.assert_within(y, wy, ref.layer_norm_tol(x, None, None, 0.0, "f32")[0], "y")
    assert float((rstd.cpu().double() / wr[:, 0] - 1).abs().max()) < 1e-4


def test_gradient_against_differences(tq):
    """The kernel's gradients against central differences of the 64-bit
    forward pass along random directions (step 1e-4: truncation below 1e-7)."""
    torch.manual_seed(0)
    x, dy = draw((6, 72), "f32", 21), draw((6, 72), "f32", 22)
    w, b = params(72, "f32", 23)
    _, mean, rstd = tq.tq_layer_norm(x.cuda(), w.cuda(), b.cuda(), 1e-5)
    dx, dw, db = (g.cpu().double() for g in tq.tq_layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd))
    f = lambda xx, ww, bb: float((ref.layer_norm(xx, ww, bb, 1e-5)[0] * dy.double()).sum())
    h = 1e-4
    for k in range(4):
        for i, grad in enumerate((dx, dw, db)):
            d = torch.randn(grad.shape, dtype=torch.float64)
            lo, hi = [x.double(), w.double(), b.double()], [x.double(), w.double(), b.double()]
            lo[i], hi[i] = lo[i] - h * d, hi[i] + h * d
            num = (f(*hi) - f(*lo)) / (2 * h)
            # binary32 gradients: 100 roundings of their terms' magnitudes
            assert abs(num - float((grad * d).sum())) < 100 * ref.U * float((grad.abs() * d.abs()).sum() + 100) + 1e-5


def test_nan_and_infinity_stay_in_their_row(tq):
    x = draw((5, 1024), "f32", 30)
    x[1, 7] = float("nan")
    x[3, 9] = float("inf")
    y, mean, rstd = (t.cpu() for t in tq.tq_layer_norm(x.cuda()))
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    good = [0, 2, 4]
    ref.assert_within(y[good], ref.layer_norm(x[good], None, None, 1e-5)[0],
                      ref.layer_norm_tol(x[good], None, None, 1e-5, "f32")[0], "y")


def test_no_rows_and_refusals(tq):
    e = torch.empty((0, 64), device="cuda")
    y, mean, rstd = tq.tq_layer_norm(e)
    assert y.shape == (0, 64)
    dx, dw, db = tq.tq_layer_norm_backward(e, e, torch.ones(64, device="cuda"), mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError):
        tq.tq_layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_layer_norm(x, torch.ones(64, device="cuda"), torch.ones(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        tq.tq_layer_norm(x.double())
    with pytest.raises(TypeError):
        tq.tq_layer_norm(x.cpu())
    with pytest.raises(tq.TQError):
        tq.tq_layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        tq.tq_layer_norm_backward(x, x, None, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_layer_norm_backward(x[:2], x, None, torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"))


def test_past_32_bit_offsets(tq):
    """[1048640, 4096] in bf16: element offsets pass 2^32."""
    rows, cols = 1048640, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    note("norm past 2^32 elements")
    y, mean, rstd = tq.tq_layer_norm(x)
    pick = [0, 1, rows // 2, 1048575, 1048576, rows - 1]
    small = x[pick].cpu()
    ref.assert_within(y[pick], ref.layer_norm(small, None, None, 1e-5)[0],
                      ref.layer_norm_tol(small, None, None, 1e-5, "bf16")[0], "y")
    dx, dw, db = tq.tq_layer_norm_backward(y, x, None, mean, rstd)
    want = ref.layer_norm_backward(y[pick].cpu(), small, None, mean[pick].cpu(), rstd[pick].cpu())[0]
    tol = ref.layer_norm_backward_tol(y[pick].cpu(), small, None, mean[pick].cpu(), rstd[pick].cpu(), "bf16", "f32")[0]
    ref.assert_within(dx[pick], want, tol, "dx")
