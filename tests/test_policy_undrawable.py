"""GPU parity of the policy loss where the token that was drawn has probability
zero, under the present policy, the old one or the reference: l = -inf is a ratio of 0
and no gradient, with a KL term an infinite loss; and a NaN among the logits is
never hidden."""
import math

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu
INF = math.inf
LO = 0.25                                               # (1 - LO) A is exact
# rho = exp(l - l') of two evaluations of one l, each off by less than 1100 units of 2^-24
# (D = 64 + 2 (38 + V / 1024) additions, 16 (1 + |z_y - m| + ln V + |l|) for its terms, at V = 140001)
ONE = 2 * 1100 * 2.0 ** -24


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def calls(tq, z, token, adv):
    """The joint call, and the two of a program with automatic differentiation."""
    def joint(**kw):
        return tq.tq_policy_loss_grad(z, token, adv, clip_low=LO, **kw)

    def apart(**kw):
        loss, logp, stats = tq.tq_policy_loss(z, token, adv, clip_low=LO, **kw)
        return loss, logp, tq.tq_policy_loss_backward(z, token, adv, logp, stats, clip_low=LO, **kw)
    return joint, apart


# rows of a thread each, held, and in parts; rows 0 and 1 draw a banned token, rows 2 and 3 have nothing to draw
def inputs(V, rows=6):
    g = torch.Generator().manual_seed(V)
    z = torch.randn((rows, V), generator=g)
    token = torch.randint(0, V, (rows,), generator=g)
    z[0, token[0]] = z[1, token[1]] = -INF
    z[2:4] = -INF
    adv = torch.tensor([2.0, -2.0, 3.0, -3.0] + [1.5, -1.5] * ((rows - 4) // 2))
    return z.cuda(), token.cuda(), adv.cuda()


@pytest.mark.parametrize("V", [6, 1003, 40001, 140001])
@pytest.mark.parametrize("rows", [6, 300])
def test_ratio_is_zero(tq, V, rows):
    if rows > 6 and V > 1003:
        rows = 6
    note("policy undrawable", rows, V)
    z, token, adv = inputs(V, rows)
    own = tq.tq_token_logp(z, token)[0]
    assert bool((own[:4] == -INF).all()) and bool(torch.isfinite(own[4:]).all())
    # -min(0, (1 - lo) A)
    want = torch.tensor([0.0, 1.5, 0.0, 2.25], device="cuda")
    for call in calls(tq, z, token, adv):
        # the present policy's own, an old policy that banned the token too, one that did not
        for old in (None, own, own.nan_to_num(neginf=-5.0)):
            loss, logp, grad = call(old_logp=old)
            assert bool((logp[:4] == -INF).all())
            assert torch.equal(loss[:4], want), (old is None, loss[:4])
            assert not grad[:4].any() and bool(torch.isfinite(grad).all())
            assert bool(((loss + adv)[4:].abs() <= ONE * adv[4:].abs()).all())
            assert bool(grad[4:].any(1).all())


@pytest.mark.parametrize("V", [6, 1003, 40001, 140001])
def test_kl_term_is_infinite(tq, V):
    z, token, adv = inputs(V)
    own = tq.tq_token_logp(z, token)[0]
    for call in calls(tq, z, token, adv):
        # a reference that banned the token too, one that did not
        for kl in (own, own.nan_to_num(neginf=-5.0)):
            for old in (None, own):
                loss, logp, grad = call(old_logp=old, ref_logp=kl, kl_coef=0.5)
                assert bool((loss[:4] == INF).all()), loss[:4]
                assert not bool(torch.isfinite(grad[:2]).all(1).any())
                assert not grad[2:4].any() and bool(torch.isfinite(grad[4:]).all())
                assert bool(((loss + adv)[4:].abs() <= ONE * adv[4:].abs()).all())


@pytest.mark.parametrize("V", [6, 1003, 40001, 140001])
def test_a_nan_is_not_hidden(tq, V):
    """A NaN logit makes its row's loss NaN with the present policy as the old one,
    as with any other; so does a NaN in old_logp or ref_logp beside l = -inf."""
    z, token, adv = inputs(V)
    z[4, V // 2] = math.nan
    nan = torch.full((6,), math.nan, device="cuda")
    for call in calls(tq, z, token, adv):
        loss, logp, grad = call()
        assert torch.isnan(logp[4]) and torch.isnan(loss[4]) and bool(torch.isnan(grad[4]).all())
        assert bool(torch.isfinite(loss[[0, 1, 2, 3, 5]]).all())
        assert bool(torch.isnan(call(old_logp=nan)[0]).all())
        assert bool(torch.isnan(call(ref_logp=nan, kl_coef=0.5)[0]).all())
