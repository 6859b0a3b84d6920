"""GPU parity of distillation where a row's logits are far from zero or far
apart: common offsets, masks of large finite values, confident students.  The
loss depends on differences of logits alone, so the bounds are those of the
other parity tests.  Rows that a workgroup holds and rows in parts."""
import math

import pytest
import torch

import llm_util as ref
from gpu_util import note
from test_parity_distill import check, draw

pytestmark = pytest.mark.gpu

# (rows, columns, type): held by 256 threads, by 512, in parts
PATHS = [(7, 2000, "f32"), (130, 17001, "f32"), (7, 70001, "f32"), (7, 2000, "bf16"), (7, 2003, "f16"),
         (7, 70001, "f16")]


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("rows,V,ft", PATHS)
@pytest.mark.parametrize("T", [1.0, 0.3])
@pytest.mark.parametrize("rest", [False, True])
def test_common_offsets(tq, rows, V, ft, T, rest):
    """Rows whose logits share a large offset, and rows of one value that a
    program uses as a mask."""
    note("distill offsets", rows, V, ft, T, rest)
    z, idx, val, tlse, dloss = draw(rows, V, 12, V + 1, "f32")
    tlse = (torch.logsumexp(val.double() / T, 1) + 0.1).float()
    top = 6.0e4 if ft == "f16" else 1.0e5
    z[0] += 1.0e3
    z[1] += 1.0e4
    z[2] -= 3.0e4
    z[3] += top
    z[4] = -65504.0
    z[5] = -6.0e4 if ft == "f16" else -1.0e9
    check(tq, z.to(ref.TORCH[ft]), idx, val, T, tlse if rest else None, dloss, ft, "T %g" % T)


def formula(z, idx, val, T, tlse, dloss):
    """Loss and gradient in 64 bits, probabilities as logarithms so that none
    underflows, and bounds of a binary32 evaluation: D roundings of a sum's depth,
    8 u of an exponential's argument, and what p_r = 1 - sum p loses (dp)."""
    s, z = 1.0 / T, z.double()
    loss, p, none = ref.distill(z, idx, val, T, tlse)
    at, V = idx.long(), z.shape[1]
    taken = torch.zeros_like(z).scatter_add_(1, at, torch.ones_like(val, dtype=torch.float64)) > 0
    pj = torch.zeros_like(z).scatter_add_(1, at, p)
    lq = torch.log_softmax(z * s, 1)
    lr = torch.logsumexp(lq.masked_fill(taken, -math.inf), 1, keepdim=True)
    big = (val.double().abs() * s).amax(1, keepdim=True) + tlse.double().abs()[:, None]
    pr = (1 - p.sum(1, keepdim=True)).clamp_min(0)
    assert bool((pr > 0.01).all())
    U, D = ref.U, 64 + 2 * ref.sum_depth(V)
    dp = (D + 8 * big) * U
    Z, q = p.sum(1, keepdim=True) + pr, lq.exp()
    lw = torch.log_softmax((z * s).masked_fill(taken, -math.inf), 1)    # lq - lr, which would lose it at 1e38
    w, size = lw.exp(), lambda v: v.abs().nan_to_num(0.0, 0.0, 0.0)
    grad = q * Z - torch.where(taken, pj, pr * w)
    tol = q * Z * ((D + 8 * size(lq)) * U + dp) + torch.where(
        taken, pj * (dp + 8 * U * size(pj.log())), w * (pr * (D + 8 * size(lw)) * U + dp))
    scale = (s * dloss.double())[:, None]
    own, lp = size(torch.where(p > 0, lq.gather(1, at), torch.zeros_like(p))), size(p.log())
    tol_l = (p * (1 + own + lp) * ((D + 8 * (own + lp)) * U + dp)).sum(1, keepdim=True)
    ratio = size(pr.log() - lr)
    tol_l = tol_l + dp * (1 + ratio) + pr * (D + 8) * U * (1 + ratio)
    # an exponential below 2^-126 is flushed before Z and the scale multiply it
    return grad * scale, tol * scale.abs() + 2.0 ** -126 * (1 + scale.abs() * (Z + pr)), loss, tol_l[:, 0] + U


def compare(tq, z, idx, val, T, tlse, dloss, ft):
    want, tol, loss, tol_l = formula(z, idx, val, T, tlse, dloss)
    tol = tol + ref.rounding(want, ft)
    dev = [t.cuda() for t in (z, idx, val, tlse, dloss)]
    l1, stats, rest = tq.tq_topk_distill(*dev[:3], temperature=T, teacher_lse=dev[3])
    g1 = tq.tq_topk_distill_backward(*dev[:3], stats, dev[4], temperature=T, teacher_lse=dev[3], rest_sum=rest)
    l2, g2 = tq.tq_topk_distill_grad(*dev[:3], dloss=dev[4], temperature=T, teacher_lse=dev[3])
    for name, l, g in (("two calls", l1, g1), ("one call", l2, g2)):
        ref.assert_within(l, loss, tol_l, name + ": loss")
        ref.assert_within(g, want, tol, name + ": gradient")


@pytest.mark.parametrize("rows,V,ft", PATHS + [(9, 7, "f32"), (170, 131072, "bf16")])
@pytest.mark.parametrize("T", [1.0, 0.1])
def test_rest_far_below_the_entries(tq, rows, V, ft, T):
    """A student that gives its entries nearly everything: the rest's mass lies
    below binary32's smallest value, and still has a logarithm and a gradient."""
    note("distill confident", rows, V, ft, T)
    K = 3 if V < 12 else 12
    z, idx, val, tlse, dloss = (t[:min(rows, 9)] for t in draw(min(rows, 9), V, K, V + 2, "f32"))
    tlse = (torch.logsumexp(val.double() / T, 1) + 0.1).float()
    inside = torch.zeros(z.shape, dtype=torch.bool).scatter_(1, idx, True)
    far = -6.0e4 if ft == "f16" else -1.0e9
    z[0] += 60.0 * inside[0]
    z[1] += 90.0 * inside[1]
    z[2, idx[2, 0]] += 300.0
    z[3] = torch.where(inside[3], z[3], torch.tensor(-1.0e4))    # masked by a finite value
    z[4] = torch.where(inside[4], z[4], torch.tensor(far))
    z[5] -= 500.0 * ~inside[5]
    z[5, torch.nonzero(~inside[5])[::2, 0]] = -math.inf          # half of the rest cannot be drawn
    z[6, idx[6, 1:]] -= 1.0e3                                    # entries far below the rest
    z[6, idx[6, 0]] += 200.0
    if V > 4096 and len(z) > 7:                                  # nothing above -inf where a wave looks first
        z[7, :4096] = -math.inf
        z[7, 4096:] -= 150.0
        idx[7] = V - 1 - torch.arange(K)
        z[7, idx[7]] += 400.0
    if rows > 9:                                                 # enough rows for the path, the same nine over and over
        z, idx, val, tlse, dloss = (t.repeat((rows + 8) // 9, *[1] * (t.dim() - 1))[:rows]
                                    for t in (z, idx, val, tlse, dloss))
    z = z.to(ref.TORCH[ft])
    if rows <= 9:
        return compare(tq, z, idx, val, T, tlse, dloss, ft)
    dev = [t.cuda() for t in (z, idx, val, tlse, dloss)]
    want, tol, loss, tol_l = formula(z[:9], idx[:9], val[:9], T, tlse[:9], dloss[:9])
    l, g = tq.tq_topk_distill_grad(*dev[:3], dloss=dev[4], temperature=T, teacher_lse=dev[3])
    for r in range(0, rows - 8, 9):
        ref.assert_within(l[r:r + 9], loss, tol_l, "loss")
        ref.assert_within(g[r:r + 9], want, tol + ref.rounding(want, ft), "gradient")


@pytest.mark.parametrize("rows,V,ft", PATHS)
def test_rest_masked_by_the_lowest_value(tq, rows, V, ft):
    note("distill lowest value", rows, V, ft)
    z, idx, val, tlse, dloss = draw(rows, V, 12, V + 3, "f32")
    inside = torch.zeros(z.shape, dtype=torch.bool).scatter_(1, idx, True)
    z = torch.where(inside, z, torch.full_like(z, torch.finfo(ref.TORCH[ft]).min)).to(ref.TORCH[ft])
    compare(tq, z, idx, val, 1.0, tlse, dloss, ft)


@pytest.mark.parametrize("rows,V,ft", PATHS)
def test_rows_that_count_nothing_have_zero_gradients(tq, rows, V, ft):
    """dloss 0, whatever the row's sums are."""
    z, idx, val, tlse, dloss = draw(rows, V, 12, V + 4, "f32")
    z[0].scatter_(0, idx[0], 5.0e4)
    z = z.to(ref.TORCH[ft])
    dev = [t.cuda() for t in (z, idx, val, tlse, torch.zeros(rows))]
    _, stats, rest = tq.tq_topk_distill(*dev[:3], teacher_lse=dev[3])
    assert not tq.tq_topk_distill_backward(*dev[:3], stats, dev[4], teacher_lse=dev[3], rest_sum=rest).any()
    assert not tq.tq_topk_distill_grad(*dev[:3], dloss=dev[4], teacher_lse=dev[3])[1].any()


def test_rest_sum_is_a_pair_per_row(tq):
    z, idx, val, tlse, dloss = (t.cuda() for t in draw(4, 64, 5, 2, "f32"))
    _, stats, rest = tq.tq_topk_distill(z, idx, val, teacher_lse=tlse)
    out = z.scatter(1, idx, -math.inf).double().cpu()
    assert torch.equal(rest[:, 0].cpu().double(), out.amax(1))
    want = (out - out.amax(1, keepdim=True)).exp().sum(1)
    ref.assert_within(rest[:, 1], want, 64 * ref.U * want, "rest_sum")
    with pytest.raises(ValueError):
        tq.tq_topk_distill_backward(z, idx, val, stats, teacher_lse=tlse, rest_sum=rest[:, 1].contiguous())
