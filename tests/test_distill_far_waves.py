"""GPU parity of distillation's held rows where two of a row's largest logits lie in
different waves: one where its wave looks first, the other further on in a wave whose
first vector is 84 to 100 (times the temperature) below it."""
import pytest
import torch

import llm_util as ref
from gpu_util import note
from test_policy_far_waves import HELD, far_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("ft,width", [(ft, i) for ft in HELD for i in range(4)])
@pytest.mark.parametrize("T", [1.0, 0.1])
@pytest.mark.parametrize("rest", [False, True])
def test_largest_logits_in_two_waves(tq, ft, width, T, rest):
    rows, V, threads = HELD[ft][width]
    note("distill far waves", rows, V, ft, T, rest)
    z, first, far = far_rows(V, threads, T, ft)
    n, K = z.shape[0], 6
    g = torch.Generator().manual_seed(2)
    # one of the two is an entry, or neither: the complement keeps one at least
    i = torch.arange(n)
    idx = 600 + 37 * torch.arange(K)[None] + i[:, None] % 17
    one = i // 3 % 3
    idx[:, 2] = torch.where(one == 0, first, torch.where(one == 1, far, idx[:, 2]))
    val = T * (1 + torch.randn((n, K), generator=g))
    tlse = (torch.logsumexp(val.double() / T, 1) + 0.3).float() if rest else None
    dloss = 0.5 + torch.rand(n, generator=g)
    want_g, tol_g, want_l = ref.distill_grad(z.double(), idx, val, T, tlse, dloss)
    tol_l = ref.distill_loss_tol(z, idx, val, T, tlse)
    # 2^x is 0 below x = -126, relative to the row's largest or to one that the row's sum holds as 1/2 or more: q is off by
    # 2^-126 / S <= 2^-125 there, and the gradient s dloss q (1 - p_r / q_r) by that times q's factor
    q = torch.softmax(z.double() / T, 1)
    qr = q.scatter(1, idx, 0.0).sum(1)
    tol_g = tol_g + 2.0 ** -125 * (dloss * (1 + (1 / qr if rest else 0)) / T)[:, None]

    row = torch.arange(rows) % n
    zd, id_, vd, dd = (t[row].cuda() for t in (z, idx, val, dloss))
    td = tlse[row].cuda() if rest else None
    loss, grad = tq.tq_topk_distill_grad(zd, id_, vd, dloss=dd, temperature=T, teacher_lse=td)
    ref.assert_within(loss[:n], want_l, tol_l, "loss, in one call")
    ref.assert_within(grad[:n], want_g, tol_g + ref.rounding(want_g, ft), "gradient, in one call")
    back = row.cuda()
    assert torch.equal(loss, loss[back]) and torch.equal(grad, grad[back])
    loss, stats, rest_sum = tq.tq_topk_distill(zd, id_, vd, temperature=T, teacher_lse=td)
    ref.assert_within(loss[:n], want_l, tol_l, "loss")
    grad = tq.tq_topk_distill_backward(zd, id_, vd, stats, dd, temperature=T, teacher_lse=td, rest_sum=rest_sum)
    ref.assert_within(grad[:n], want_g, tol_g + ref.rounding(want_g, ft), "gradient")
