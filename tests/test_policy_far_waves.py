"""GPU parity of the policy loss's held rows where two of a row's largest logits
lie in different waves: one where its wave looks first, the other further on in a
wave whose first vector is 84 to 100 (times the temperature) below it.  Such a wave's
own sum is near binary32's largest, and what scales it to the row near its smallest."""
import pytest
import torch

import llm_util as ref
import policy_util as pu
from gpu_util import note

pytestmark = pytest.mark.gpu
LO, HI, BETA = 0.2, 0.28, 0.1
GAPS = (84.0, 86.0, 87.3, 87.6, 87.8, 88.0, 88.3, 88.6, 89.0, 100.0)

# (rows, columns, threads per row): every width of a held row, at the fewest rows that are held
HELD = {"f32": [(90, 8000, 256), (90, 16001, 256), (128, 32003, 512), (448, 40005, 1024)],
        "bf16": [(90, 8192, 256), (90, 32003, 256), (128, 65001, 512), (160, 80003, 1024)]}


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def far_rows(V, threads, T, ft):
    """(logits, the columns of the two): 90 rows of every gap, difference and place."""
    g = torch.Generator().manual_seed(V)
    n = 9 * len(GAPS)
    z = 0.1 * T * torch.randn((n, V), generator=g)
    first = torch.arange(n) % 512                          # wave 0's first vector
    # the second vector of wave 1, or the last whole one of wave 2
    far = torch.where(torch.arange(n) % 2 == 0, 8 * threads + 512 + torch.arange(n),
                      V // 8 // threads * 8 * threads - 8 * threads + 1024 + torch.arange(n))
    gap = torch.tensor(GAPS).repeat_interleave(9)
    apart = torch.tensor([-0.4, 0.0, 0.5]).repeat(n // 3)
    z.scatter_(1, first[:, None], T * gap[:, None])
    z.scatter_(1, far[:, None], T * (gap + apart)[:, None])
    return z.to(ref.TORCH[ft]), first, far


@pytest.mark.parametrize("ft,width", [(ft, i) for ft in HELD for i in range(4)])
@pytest.mark.parametrize("T", [1.0, 0.1])
def test_largest_logits_in_two_waves(tq, ft, width, T):
    rows, V, threads = HELD[ft][width]
    note("policy far waves", rows, V, ft, T)
    z, first, far = far_rows(V, threads, T, ft)
    n = z.shape[0]
    i = torch.arange(n)
    token = torch.where(i // 3 % 3 == 0, first, torch.where(i // 3 % 3 == 1, far, torch.full_like(far, 1500)))
    g = torch.Generator().manual_seed(1)
    l = pu.logp(z, token, T)[1]
    drift = 0.1 * torch.rand(n, generator=g, dtype=torch.float64)          # inside both clips
    old, kl = (l - drift).float(), (l + 0.2 * drift).float()
    adv, dloss = torch.randn(n, generator=g), 0.5 + torch.rand(n, generator=g)
    tl = pu.logp_tol(z, token, T)
    t_loss, t_slope = pu.tolerances(l, tl, adv, old, kl, BETA)
    want = pu.loss(l, adv, old, kl, LO, HI, BETA)
    slope = pu.slope(l, adv, old, kl, LO, HI, BETA)
    grad, t_grad = pu.gradient(z, token, T, slope * dloss, t_slope * dloss, ft)
    # 2^x is 0 below x = -126, relative to the row's largest or to one that the row's sum holds as 1/2 or more: q is off by
    # 2^-126 / S <= 2^-125 there, and the gradient by that times its factor
    t_grad = t_grad + 2.0 ** -125 * (slope * dloss).abs()[:, None] / T

    row = torch.arange(rows) % n
    zd, td, ad, od, kd, dd = (t[row].cuda() for t in (z, token, adv, old, kl, dloss))
    how = dict(old_logp=od, ref_logp=kd, clip_low=LO, clip_high=HI, kl_coef=BETA, temperature=T)
    loss, logp, dz = tq.tq_policy_loss_grad(zd, td, ad, dloss=dd, **how)
    ref.assert_within(logp[:n], l, tl, "logp, in one call")
    ref.assert_within(loss[:n], want, t_loss, "loss, in one call")
    ref.assert_within(dz[:n], grad, t_grad, "gradient, in one call")
    back = row.cuda()
    assert torch.equal(logp, logp[back]) and torch.equal(loss, loss[back]) and torch.equal(dz, dz[back])
    loss, logp, stats = tq.tq_policy_loss(zd, td, ad, **how)
    ref.assert_within(logp[:n], l, tl, "logp")
    dz = tq.tq_policy_loss_backward(zd, td, ad, logp, stats, dloss=dd, **how)
    ref.assert_within(dz[:n], grad, t_grad, "gradient")
