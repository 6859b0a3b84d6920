"""GPU parity of the policy loss where the ratio leaves binary32: without an
advantage the clipped term and its gradient are 0 all the same, as 64 bits have it."""
import math

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("V", [6, 1003, 140001])
def test_ratio_overflows_without_an_advantage(tq, V):
    note("policy overflow", V)
    g = torch.Generator().manual_seed(V)
    rows = 6
    z, token = torch.randn((rows, V), generator=g).cuda(), torch.randint(0, V, (rows,), generator=g).cuda()
    l = tq.tq_token_logp(z, token)[0]
    old = l - torch.tensor([100.0, 500.0, math.inf, 100.0, 0.0, math.nan], device="cuda")
    adv = torch.tensor([0.0, -0.0, 0.0, 1.0, 0.0, 0.0], device="cuda")
    loss, logp, both = tq.tq_policy_loss_grad(z, token, adv, old_logp=old, clip_high=0.25)
    loss2, logp2, stats = tq.tq_policy_loss(z, token, adv, old_logp=old, clip_high=0.25)
    back = tq.tq_policy_loss_backward(z, token, adv, logp2, stats, old_logp=old, clip_high=0.25)
    for lo, grad in ((loss, both), (loss2, back)):
        assert not lo[[0, 1, 2, 4]].any() and lo[3] == -1.25 and torch.isnan(lo[5])
        assert not grad[:5].any() and bool(torch.isnan(grad[5]).all())
    # the KL term beside it is what it is alone
    a = tq.tq_policy_loss_grad(z[:3], token[:3], adv[:3], old_logp=old[:3], ref_logp=l[:3] + 0.5, kl_coef=0.3)
    b = tq.tq_policy_loss_grad(z[:3], token[:3], adv[:3], ref_logp=l[:3] + 0.5, kl_coef=0.3)
    assert all(torch.equal(p, q) for p, q in zip(a, b)) and bool((a[0] > 0).all())
