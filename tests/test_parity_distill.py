"""GPU parity: distillation from a teacher's top logits against its 64-bit
definition: loss, the saved statistics, the gradient by both ways, padding
entries, banned tokens, rows that a mask leaves empty, repeated columns."""
import math

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


def draw(rows, V, K, seed, ft, padded=False, idx=torch.int64, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    order = torch.stack([torch.randperm(V, generator=g)[:min(K, V)] for _ in range(rows)])
    if K > V:
        order = torch.cat([order, torch.full((rows, K - V), -1, dtype=torch.int64)], 1)
    val = (3 + 2 * torch.randn((rows, K), generator=g)).sort(1, descending=True).values
    z = 2 * sharp * torch.randn((rows, V), generator=g)
    z.scatter_add_(1, order.clamp_min(0), torch.where(order >= 0, 0.8 * val, torch.zeros_like(val)))
    if padded:
        left = torch.randint(0, K + 1, (rows, 1), generator=g)
        order = torch.where(torch.arange(K)[None] < left, order, torch.full_like(order, -1))
    tlse = torch.logsumexp(val.double(), 1) + 0.05 + 0.3 * torch.rand(rows, generator=g, dtype=torch.float64)
    dloss = 0.5 + torch.rand(rows, generator=g)
    return z.to(ref.TORCH[ft]), order.to(idx), val, tlse.float(), dloss


def check(tq, z, idx, val, T, tlse, dloss, ft, what=""):
    zd, id_, vd = z.cuda(), idx.cuda(), val.cuda()
    td = None if tlse is None else tlse.cuda()
    dd = None if dloss is None else dloss.cuda()
    want_g, tol_g, want_l = ref.distill_grad(z.double(), idx, val, T, tlse, dloss)
    tol_l = ref.distill_loss_tol(z, idx, val, T, tlse)
    loss, stats, rest = tq.tq_topk_distill(zd, id_, vd, temperature=T, teacher_lse=td)
    ref.assert_within(loss, want_l, tol_l, what + " loss")
    grad = tq.tq_topk_distill_backward(zd, id_, vd, stats, dd, temperature=T, teacher_lse=td, rest_sum=rest)
    tol = tol_g + ref.rounding(want_g, ft)
    ref.assert_within(grad, want_g, tol, what + " gradient")
    loss2, grad2 = tq.tq_topk_distill_grad(zd, id_, vd, dloss=dd, temperature=T, teacher_lse=td)
    ref.assert_within(loss2, want_l, tol_l, what + " loss in one call")
    ref.assert_within(grad2, want_g, tol, what + " gradient in one call")
    return loss, grad, loss2, grad2


# below one vector, vector and part boundaries, a row held by each workgroup size, longer than any holds
@pytest.mark.parametrize("rows,V,K", [(1, 1, 1), (3, 5, 4), (2, 8, 8), (5, 9, 3), (2, 100, 7), (9, 4096, 16),
                                      (3, 4097, 33), (2, 8200, 1024), (1, 33001, 64), (130, 7, 2), (130, 63, 5),
                                      (129, 8191, 9), (128, 8209, 20), (128, 20001, 300)])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("ft", ["f32", "bf16", "f16"])
def test_sizes(tq, rows, V, K, rest, ft):
    note("distill", rows, V, K, rest, ft)
    z, idx, val, tlse, dloss = draw(rows, V, K, V + K, ft)
    check(tq, z, idx, val, 1.0, tlse if rest else None, dloss, ft)


@pytest.mark.parametrize("rows", [131, 170])
@pytest.mark.parametrize("V,ft", [(40003, "bf16"), (65536, "f16"), (70001, "bf16"), (98304, "bf16"), (131072, "bf16"),
                                  (131001, "f16"), (50001, "f32"), (65544, "f32"), (140000, "bf16")])
def test_long_rows(tq, rows, V, ft):
    long_rows(tq, rows, V, ft)


def test_long_binary32_rows_of_two_rounds(tq):
    long_rows(tq, 450, 40003, "f32")


def long_rows(tq, rows, V, ft):
    note("distill long", rows, V, ft)
    z, idx, val, tlse, dloss = draw(rows, V, 40, V, ft)
    pick = [0, 1, 64, 129, 130]
    zd, id_, vd, td = z.cuda(), idx.cuda(), val.cuda(), tlse.cuda()
    loss, grad = tq.tq_topk_distill_grad(zd, id_, vd, dloss=dloss.cuda(), teacher_lse=td)
    loss2, stats, rest = tq.tq_topk_distill(zd, id_, vd, teacher_lse=td)
    grad2 = tq.tq_topk_distill_backward(zd, id_, vd, stats, dloss.cuda(), teacher_lse=td, rest_sum=rest)
    want_g, tol_g, want_l = ref.distill_grad(z[pick].double(), idx[pick], val[pick], 1.0, tlse[pick], dloss[pick])
    tol_l = ref.distill_loss_tol(z[pick], idx[pick], val[pick], 1.0, tlse[pick])
    for l, g in ((loss, grad), (loss2, grad2)):
        ref.assert_within(l[pick], want_l, tol_l, "loss")
        ref.assert_within(g[pick], want_g, tol_g + ref.rounding(want_g, ft), "gradient")


@pytest.mark.parametrize("T", [0.5, 1.0, 2.0, 7.0])
@pytest.mark.parametrize("rest", [False, True])
def test_temperature_types_and_padding(tq, T, rest):
    for rows in (6, 140):
        z, idx, val, tlse, dloss = draw(rows, 1003, 12, 17, "bf16", padded=True, idx=torch.int32)
        val = val.to(torch.bfloat16)
        tlse = (torch.logsumexp(val.double() / T, 1) + 0.1).float()
        check(tq, z, idx, val, T, tlse if rest else None, dloss, "bf16")
        check(tq, z, idx, val.float().to(torch.float16), T, tlse if rest else None, None, "bf16")


# held rows, and rows in parts
@pytest.mark.parametrize("rows,V", [(8, 2000), (150, 2000), (8, 70001), (8, 140000)])
@pytest.mark.parametrize("rest", [False, True])
def test_masks_infinities_and_empty_rows(tq, rows, V, rest):
    z, idx, val, tlse, dloss = draw(rows, V, 10, 3, "f32")
    low = torch.finfo(torch.float32).min
    z[0, 500:] = -math.inf                              # banned tokens, some of them the teacher's
    idx[1] = -1                                         # no entries
    idx[2, 3:] = V                                      # past the vocabulary: padding
    idx[2, 5] = 1 << 40                                 # far past it
    z[3] = -math.inf                                    # nothing can be drawn
    z[4, 100:] = low                                    # masked by the type's lowest value
    idx[4] = torch.arange(10)
    z[5] = low                                          # a whole row of it: uniform
    val[6, 2:] = -math.inf                              # entries of no weight
    val[7] = -math.inf                                  # nothing but such
    tlse[7] = 0.5
    loss, grad, loss2, grad2 = check(tq, z, idx, val, 1.0, tlse if rest else None, dloss, "f32")
    for l, g in ((loss, grad), (loss2, grad2)):
        assert l[1] == 0 and not g[1].any()
        assert torch.isinf(l[3]) and l[3] > 0 and not g[3].any()
        assert not torch.isnan(g).any()
    if not rest:
        assert loss[7] == 0 and not grad[7].any() and not grad2[7].any()


@pytest.mark.parametrize("rows,V", [(4, 777), (130, 777), (4, 70001)])
def test_nan_stays_in_its_row_and_empty_rows_ignore_it(tq, rows, V):
    z, idx, val, tlse, dloss = draw(rows, V, 6, 8, "f32")
    z[1, 5] = math.nan
    z[2, 9] = math.nan
    idx[2] = -1
    for loss, grad in (tq.tq_topk_distill_grad(z.cuda(), idx.cuda(), val.cuda()),):
        assert torch.isnan(loss[1]) and torch.isnan(grad[1]).all()
        assert loss[2] == 0 and not grad[2].any()
        assert torch.isfinite(loss[[0, 3]]).all() and torch.isfinite(grad[[0, 3]]).all()
    loss, stats, _ = tq.tq_topk_distill(z.cuda(), idx.cuda(), val.cuda())
    grad = tq.tq_topk_distill_backward(z.cuda(), idx.cuda(), val.cuda(), stats)
    assert torch.isnan(loss[1]) and torch.isnan(grad[1]).all() and loss[2] == 0 and not grad[2].any()


@pytest.mark.parametrize("rows,V", [(3, 300), (200, 300), (3, 70001)])
@pytest.mark.parametrize("rest", [False, True])
def test_repeated_columns_add_up(tq, rows, V, rest):
    z, idx, val, tlse, dloss = draw(rows, V, 9, 5, "f32")
    idx[:, 4] = idx[:, 0]
    idx[:, 7] = idx[:, 0]
    idx[:, 8] = idx[:, 3]
    a = check(tq, z, idx, val, 1.0, tlse if rest else None, dloss, "f32")
    b = check(tq, z, idx, val, 1.0, tlse if rest else None, dloss, "f32")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("rows,V", [(5, 5000), (140, 5000), (140, 1001), (3, 70001)])
def test_strides_and_in_place(tq, rows, V):
    z, idx, val, tlse, dloss = draw(rows, V, 11, 6, "bf16")
    wide = torch.full((rows, V + 5), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + V] = z.cuda()
    args = dict(teacher_lse=tlse.cuda(), dloss=dloss.cuda())
    loss, grad = tq.tq_topk_distill_grad(z.cuda(), idx.cuda(), val.cuda(), **args)
    loss2, grad2 = tq.tq_topk_distill_grad(wide[:, 2:2 + V], idx.cuda(), val.cuda(), **args)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)
    loss3, grad3 = tq.tq_topk_distill_grad(wide[:, 2:2 + V], idx.cuda(), val.cuda(), inplace=True, **args)
    assert torch.equal(loss, loss3) and torch.equal(grad, grad3)
    assert torch.equal(wide[:, 2:2 + V], grad) and bool((wide[:, :2] == 9).all()) and bool((wide[:, 2 + V:] == 9).all())


def test_student_equal_to_its_teacher(tq):
    """Every entry given and the student the teacher itself: loss and gradient
    vanish to rounding (a difference of logarithms would not)."""
    g = torch.Generator().manual_seed(1)
    z = 4 * torch.randn((150, 64), generator=g)
    val, idx = z.sort(1, descending=True)
    loss, grad = tq.tq_topk_distill_grad(z.cuda(), idx.cuda(), val.cuda())
    assert float(loss.abs().max()) < 1e-6 and float(grad.abs().max()) < 1e-6
    tlse = torch.logsumexp(z.double(), 1).float()
    loss, grad = tq.tq_topk_distill_grad(z.cuda(), idx[:, :20].contiguous().cuda(), val[:, :20].contiguous().cuda(),
                                         teacher_lse=tlse.cuda())
    assert float(loss.abs().max()) < 3e-6 and float(grad.abs().max()) < 3e-6


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences(tq, rest):
    """Central differences of the 64-bit loss along random directions (step
    1e-4: truncation below 1e-7)."""
    z, idx, val, tlse, dloss = draw(5, 90, 8, 12, "f32")
    t = tlse if rest else None
    _, grad = tq.tq_topk_distill_grad(z.cuda(), idx.cuda(), val.cuda(), dloss=dloss.cuda(), temperature=1.5,
                                      teacher_lse=None if t is None else t.cuda())
    grad = grad.cpu().double()
    f = lambda zz: float((ref.distill(zz, idx, val, 1.5, t)[0] * dloss.double()).sum())
    torch.manual_seed(4)
    h = 1e-4
    for _ in range(5):
        d = torch.randn(z.shape, dtype=torch.float64)
        num = (f(z.double() + h * d) - f(z.double() - h * d)) / (2 * h)
        assert abs(num - float((grad * d).sum())) < 1e-6 + 300 * ref.U * float(d.abs().sum())


def test_refusals(tq):
    z, idx, val, tlse, dloss = (t.cuda() for t in draw(4, 64, 5, 2, "f32"))
    call = tq.tq_topk_distill_grad
    with pytest.raises(tq.TQError):
        call(z, idx, val, temperature=0.0)
    with pytest.raises(tq.TQError):
        call(z, idx, val, temperature=float("nan"))
    with pytest.raises(TypeError):
        call(z, idx.float(), val)
    with pytest.raises(ValueError):
        call(z, idx[:3], val)
    with pytest.raises(ValueError):
        call(z, idx, val[:, :4])
    with pytest.raises(ValueError):
        call(z, idx, val, teacher_lse=tlse[:3])
    with pytest.raises(ValueError):
        call(z, idx, val, dloss=dloss.double())
    with pytest.raises(ValueError):
        call(z.t(), idx.new_zeros((64, 5)), val.new_zeros((64, 5)), inplace=True)
    with pytest.raises(tq.TQError):
        call(z, idx.new_zeros((4, 1025)), val.new_zeros((4, 1025)))
    with pytest.raises(tq.TQError):
        call(z, idx[:, :0], val[:, :0])
    _, stats, rest = tq.tq_topk_distill(z, idx, val)
    with pytest.raises(ValueError):
        tq.tq_topk_distill_backward(z, idx, val, stats, teacher_lse=tlse)
    e = z[:0]
    loss, grad = call(e, idx[:0], val[:0])
    assert loss.shape == (0,) and grad.shape == (0, 64)
