"""GPU parity: a token's log-probability and the clipped policy loss against their
64-bit definitions: loss, log-probability, the saved statistics, the gradient by
both ways, rows that count nowhere, banned tokens, logits far from zero."""
import math

import pytest
import torch

import llm_util as ref
import policy_util as pu
from gpu_util import note

pytestmark = pytest.mark.gpu
LO, HI, BETA = 0.2, 0.28, 0.1


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def draw(rows, V, seed, ft, T=1.0, padded=False, idx=torch.int64, kl=True, old=True):
    g = torch.Generator().manual_seed(seed)
    token = torch.randint(0, V, (rows,), generator=g)
    z = 2 * torch.randn((rows, V), generator=g)
    z.scatter_add_(1, token[:, None], 3 + 2 * torch.randn((rows, 1), generator=g))
    z = z.to(ref.TORCH[ft])
    lq, l, _, _, _ = pu.logp(z, token, T)
    drift = 0.2 * torch.randn(rows, generator=g, dtype=torch.float64)
    rho = drift.exp()
    edge = torch.minimum((rho - (1 - LO)).abs(), (rho - (1 + HI)).abs()) < 1e-3
    # far enough from a clip's edge that binary32 cannot mistake its side
    old_logp = (l - torch.where(edge, 0.5 * drift, drift)).float() if old else None
    ref_logp = (l + 0.3 * torch.randn(rows, generator=g, dtype=torch.float64)).float() if kl else None
    adv, dloss = torch.randn(rows, generator=g), 0.5 + torch.rand(rows, generator=g)
    if padded:
        out = torch.tensor([-1, V, -5, 2 ** 31 - 1])[torch.randint(0, 4, (rows,), generator=g)]
        token = torch.where(torch.rand(rows, generator=g) < 0.4, out, token)
    return z, token.to(idx), adv, old_logp, ref_logp, dloss


def check(tq, z, token, adv, old, kl, dloss, ft, T=1.0, beta=BETA, what=""):
    dev = [None if t is None else t.cuda() for t in (z, token, adv, old, kl, dloss)]
    zd, td, ad, od, kd, dd = dev
    how = dict(old_logp=od, ref_logp=kd, clip_low=LO, clip_high=HI, kl_coef=beta, temperature=T)
    lq, l, here, at, dead = pu.logp(z, token, T)
    tl = pu.logp_tol(z, token, T).masked_fill(~here, 0)
    want = pu.loss(l, adv, old, kl, LO, HI, beta).masked_fill(~here, 0)
    t_loss, t_slope = pu.tolerances(l, tl, adv, old, kl, beta)
    slope = pu.slope(l, adv, old, kl, LO, HI, beta)
    g = torch.ones_like(l) if dloss is None else dloss.double()

    loss, logp, stats = tq.tq_policy_loss(zd, td, ad, **how)
    ref.assert_within(logp, l, tl, what + " logp")
    ref.assert_within(loss, want, t_loss.masked_fill(~here, 0), what + " loss")
    counts = here & ~dead
    ref.assert_within(stats[:, 0].cpu()[counts], z.double().amax(1)[counts], 0 * l[counts], what + " largest")
    S = (lq - lq.amax(1, keepdim=True)).exp().sum(1)[counts]
    D = 64 + 2 * ref.sum_depth(z.shape[1])
    ref.assert_within(stats[:, 1].cpu()[counts], S, S * ref.U * (D + 16 * math.log(z.shape[1]) + 16), what + " sum")
    assert torch.equal(stats[:, 0].cpu()[~here], torch.full(((~here).sum(),), -math.inf)) and not stats[:, 1].cpu()[~here].any()

    grad, t_grad = pu.gradient(z, token, T, slope * g, t_slope * g.abs(), ft)
    back = tq.tq_policy_loss_backward(zd, td, ad, logp, stats, dloss=dd, **how)
    ref.assert_within(back, grad, t_grad, what + " gradient")
    loss2, logp2, both = tq.tq_policy_loss_grad(zd, td, ad, dloss=dd, **how)
    ref.assert_within(logp2, l, tl, what + " logp, in one call")
    ref.assert_within(loss2, want, t_loss.masked_fill(~here, 0), what + " loss, in one call")
    ref.assert_within(both, grad, t_grad, what + " gradient, in one call")
    alone, stats2 = tq.tq_token_logp(zd, td, T)
    assert torch.equal(alone, logp) and torch.equal(stats2, stats)
    g1, t1 = pu.gradient(z, token, T, g, 0 * g, ft)
    ref.assert_within(tq.tq_token_logp_backward(zd, td, stats, dd, T), g1, t1, what + " gradient of logp")
    return loss, logp, back, both


# every kernel: rows held by 256 threads (short, long), in parts, a workgroup per row; widths off every vector and part
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 5), (2, 7), (1, 8), (5, 9), (4, 1000), (33, 1003), (2, 8192), (3, 8195),
                                    (5, 32000), (2, 32771), (300, 1), (300, 6), (257, 515), (300, 8200), (260, 9001),
                                    (1, 131072), (3, 131001), (130, 40001), (2, 200003), (1, 300000), (1100, 64)])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_sizes(tq, rows, V, ft):
    note("policy", rows, V, ft)
    check(tq, *draw(rows, V, rows + V, ft, padded=rows > 2), ft, what="%dx%d %s" % (rows, V, ft))


# rows that fill a CU each, held from 5/8 (7/8) of a round on, more rows than workgroups
@pytest.mark.parametrize("rows,V,ft", [(165, 70001, "bf16"), (160, 131072, "f16"), (450, 40003, "f32"), (300, 20001, "f32"),
                                       (520, 33001, "f16"), (1030, 9003, "bf16"), (2100, 4100, "f32"), (4100, 1001, "bf16")])
def test_many_rows(tq, rows, V, ft):
    note("policy, many rows", rows, V, ft)
    check(tq, *draw(rows, V, V, ft, padded=True), ft, what="%dx%d" % (rows, V))


@pytest.mark.parametrize("T", [0.5, 1.7])
@pytest.mark.parametrize("kl,old", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,V", [(40, 3001), (3, 140001)])
def test_terms(tq, T, kl, old, idx, rows, V):
    check(tq, *draw(rows, V, 7, "f32", T, True, idx, kl, old), "f32", T)


def test_no_rows_and_nobody(tq):
    f = lambda *s: torch.ones(s, device="cuda")
    none = torch.full((4,), -1, device="cuda")
    for V in (5, 100, 140000):
        nan = float("nan") * f(4, V)
        loss, logp, stats = tq.tq_policy_loss(nan, none, f(4), ref_logp=f(4), kl_coef=1.0)
        assert not loss.any() and not logp.any()
        assert not tq.tq_policy_loss_backward(nan, none, f(4), logp, stats).any()
        loss, logp, grad = tq.tq_policy_loss_grad(nan, none, float("nan") * f(4))
        assert not loss.any() and not logp.any() and not grad.any()
        assert not tq.tq_token_logp_backward(nan, none, stats, float("nan") * f(4)).any()
    loss, logp, grad = tq.tq_policy_loss_grad(f(0, 9), none[:0], f(0))
    assert loss.shape == logp.shape == (0,) and grad.shape == (0, 9)


@pytest.mark.parametrize("rows,V", [(3, 1003), (2, 40001), (300, 3001), (1, 140001)])
@pytest.mark.parametrize("shift", [1e4, -1e4, 3e6, -1e9])
def test_common_offsets(tq, rows, V, shift):
    """Logits far from zero: what binary32 logits there say is met to their own
    spacing's accuracy, since all arithmetic is on differences."""
    z, token, adv, old, kl, dloss = draw(rows, V, 11, "f32")
    z = z + shift
    l = pu.logp(z, token, 1.0)[1]
    old = (l - 0.1).float()
    check(tq, z, token, adv, old, (l + 0.2).float(), dloss, "f32", what="offset %g" % shift)


@pytest.mark.parametrize("rows,V", [(4, 1003), (3, 33001), (300, 2000), (2, 131072), (2, 150001), (170, 70001)])
@pytest.mark.parametrize("ft", ["bf16", "f32"])
def test_far_apart(tq, rows, V, ft):
    """The row's largest logits lie where no wave looks first, or everything but a
    few columns is masked by the type's lowest value, -inf, or a large finite one."""
    z, token, adv, _, _, dloss = draw(rows, V, 5, ft, kl=False, old=False)
    low = torch.finfo(z.dtype).min
    for k, mask in enumerate((low, -math.inf, -1e4, -1e9)):
        y = z.clone()
        y[:, :V // 2] = mask
        y[:, V - 3:] = y[:, V - 3:] + 60
        y.scatter_(1, token[:, None], torch.full((rows, 1), 1.0).to(z.dtype))
        l = pu.logp(y, token, 1.0)[1]
        check(tq, y, token, adv, (l + 0.05).float(), (l - 0.1).float(), dloss, ft, what="mask %g" % mask)


@pytest.mark.parametrize("V", [6, 1003, 40001, 140001])
@pytest.mark.parametrize("rows", [3, 300])
def test_what_cannot_be_drawn(tq, V, rows):
    inf = math.inf
    if rows * V > 2e7:
        rows = 130
    z, token, adv, old, kl, dloss = draw(rows, V, 3, "f32")
    z[0] = -inf                                          # a row of nothing but -inf
    z[1, token[1]] = -inf                                # a banned token that was drawn all the same
    dev = [t.cuda() for t in (z, token, adv, old, kl, dloss)]
    for call in (lambda **k: tq.tq_policy_loss_grad(*dev[:3], **k),
                 lambda **k: (lambda lo, lp, st: (lo, lp, tq.tq_policy_loss_backward(*dev[:3], lp, st, **k)))(
                     *tq.tq_policy_loss(*dev[:3], **k))):
        loss, logp, grad = call(old_logp=dev[3])
        assert logp[0] == -inf and logp[1] == -inf and torch.isfinite(logp[2:]).all()
        assert torch.isfinite(loss).all() and not grad[:2].any() and torch.isfinite(grad).all()
        loss, logp, grad = call(old_logp=dev[3], ref_logp=dev[4], kl_coef=0.1)
        assert loss[0] == inf and loss[1] == inf and torch.isfinite(loss[2:]).all()
        assert not grad[0].any() and not torch.isfinite(grad[1]).all() and torch.isfinite(grad[2:]).all()


@pytest.mark.parametrize("V", [5, 1003, 32001, 140001])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_stays_in_its_row(tq, V, bad):
    z, token, adv, old, kl, dloss = draw(5, V, 9, "f32")
    want = tq.tq_policy_loss_grad(z.cuda(), token.cuda(), adv.cuda(), old_logp=old.cuda())
    z[2, V // 2] = bad
    got = tq.tq_policy_loss_grad(z.cuda(), token.cuda(), adv.cuda(), old_logp=old.cuda())
    keep = torch.tensor([0, 1, 3, 4], device="cuda")
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(got[1][2]) and torch.isnan(got[2][2]).any()
    adv[1] = math.nan
    loss, logp, grad = tq.tq_policy_loss_grad(z.cuda(), token.cuda(), adv.cuda(), old_logp=old.cuda())
    assert torch.isnan(loss[1]) and torch.isnan(grad[1]).all() and torch.equal(grad[keep[[0, 2, 3]]], want[2][keep[[0, 2, 3]]])


@pytest.mark.parametrize("rows,V,ft", [(3, 5, "f32"), (9, 1003, "bf16"), (300, 2003, "f16"), (2, 40001, "f32"),
                                       (3, 131001, "f16"), (165, 70001, "bf16"), (2, 300001, "bf16")])
def test_gradient_over_the_logits(tq, rows, V, ft):
    note("policy in place", rows, V, ft)
    z, token, adv, old, kl, dloss = (t.cuda() for t in draw(rows, V, 13, ft, padded=True))
    how = dict(dloss=dloss, old_logp=old, ref_logp=kl, kl_coef=BETA)
    want = tq.tq_policy_loss_grad(z, token, adv, **how)
    got = tq.tq_policy_loss_grad(z, token, adv, inplace=True, **how)
    assert got[2].data_ptr() == z.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,V", [(9, 1003), (300, 515), (2, 40001), (2, 140001)])
def test_strided_logits(tq, rows, V):
    z, token, adv, old, kl, dloss = (t.cuda() for t in draw(rows, V, 17, "bf16"))
    wide = torch.full((rows, V + 11), float("nan"), dtype=z.dtype, device="cuda")
    view = wide[:, 5:5 + V]
    view.copy_(z)
    want = tq.tq_policy_loss_grad(z, token, adv, old_logp=old)
    got = tq.tq_policy_loss_grad(view, token, adv, old_logp=old)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    l, stats = tq.tq_token_logp(view, token)
    assert torch.equal(l, tq.tq_token_logp(z, token)[0])
    assert torch.equal(tq.tq_token_logp_backward(view, token, stats), tq.tq_token_logp_backward(z, token, stats))
    got = tq.tq_policy_loss_grad(view, token, adv, old_logp=old, inplace=True)
    assert torch.equal(view, want[2]) and torch.isnan(wide[:, :5]).all() and torch.isnan(wide[:, 5 + V:]).all()


@pytest.mark.parametrize("rows,V", [(1, 5), (3, 4097), (9, 131001), (128, 70001), (600, 9001)])
def test_keeps_inside(tq, rows, V):
    note("policy, guarded buffers", rows, V)
    z, token, adv, old, kl, dloss = (t.cuda() for t in draw(rows, V, 19, "f32", padded=True))
    want = tq.tq_policy_loss(z, token, adv, old_logp=old)
    want_g = tq.tq_policy_loss_grad(z, token, adv, old_logp=old)
    n, G = tq.tq_policy_loss_workspace_bytes(rows, V), 4096
    bufs = [torch.full((G + b + G,), 255, dtype=torch.uint8, device="cuda") for b in (n, 4 * rows, 4 * rows, 8 * rows, 4 * rows * V)]
    ws, loss, logp, stats, grad = (b.data_ptr() + G for b in bufs)
    head = (z.data_ptr(), 0, rows, V, V, token.data_ptr(), 64, adv.data_ptr(), old.data_ptr(), None, 0.2, 0.2, 0.0, 1.0)
    st = torch.cuda.current_stream().cuda_stream

    def inside(k):
        return bufs[k][G:-G].view(torch.float32)
    assert 0 == tq._lib.tq_policy_loss(*head, loss, logp, stats, ws, n, st)
    assert torch.equal(inside(1), want[0]) and torch.equal(inside(2), want[1]) and torch.equal(inside(3), want[2].view(-1))
    assert 0 == tq._lib.tq_policy_loss_grad(*head, None, loss, logp, grad, V, ws, n, st)
    assert torch.equal(inside(1), want_g[0]) and torch.equal(inside(4), want_g[2].view(-1))
    for b in bufs:
        assert bool((b[:G] == 255).all()) and bool((b[-G:] == 255).all())


def test_gradient_against_differences(tq):
    """The gradient against central differences of the loss's definition in 64 bits
    (step 1e-5: truncation and rounding below 1e-8) and against its differentiation, on
    both sides of the clips; binary32 is within a hundred roundings of values below 2."""
    rows, V, h = 12, 24, 1e-5
    z, token, adv, old, kl, _ = draw(rows, V, 23, "f32")
    l = pu.logp(z, token, 1.3)[1]
    old = (l - torch.linspace(-0.6, 0.6, rows, dtype=torch.float64)).float()
    kl = (l + 0.2).float()
    _, _, grad = tq.tq_policy_loss_grad(z.cuda(), token.cuda(), adv.cuda(), old_logp=old.cuda(), ref_logp=kl.cuda(),
                                        clip_low=LO, clip_high=HI, kl_coef=BETA, temperature=1.3)

    def f(z):
        lq = torch.log_softmax(z / 1.3, 1).gather(1, token[:, None])[:, 0]
        return pu.loss(lq, adv, old, kl, LO, HI, BETA)
    zd, num = z.double(), torch.zeros(rows, V, dtype=torch.float64)
    for j in range(V):
        e = torch.zeros(V, dtype=torch.float64)
        e[j] = h
        num[:, j] = (f(zd + e) - f(zd - e)) / (2 * h)
    close = 100 * ref.U * 2
    assert float((grad.cpu().double() - num).abs().max()) < 1e-8 + close
    a = z.double().requires_grad_()
    f(a).sum().backward()
    assert float((grad.cpu().double() - a.grad).abs().max()) < close


def test_clips(tq):
    """Loss and gradient on a row of two columns, where l and the ratio are known."""
    z = torch.zeros((6, 2)).cuda()
    token = torch.tensor([0, 0, 0, 0, 1, 1]).cuda()
    rho = torch.tensor([1.5, 1.5, 0.5, 0.5, 1.0, 1.1])
    adv = torch.tensor([2.0, -2.0, 2.0, -2.0, 1.0, 1.0])
    old = (math.log(0.5) - rho.double().log()).float()
    loss, logp, grad = tq.tq_policy_loss_grad(z, token, adv.cuda(), old_logp=old.cuda(), clip_low=0.2, clip_high=0.3)
    want = torch.tensor([-2.6, 3.0, -1.0, 1.6, -1.0, -1.1])
    k = torch.tensor([0.0, 3.0, -1.0, 0.0, -1.0, -1.1])
    assert torch.allclose(loss.cpu(), want, rtol=1e-6) and torch.allclose(logp.cpu(), torch.full((6,), math.log(0.5)), rtol=1e-6)
    at = grad.cpu().gather(1, token.cpu()[:, None])[:, 0]
    assert torch.allclose(at, 0.5 * k, rtol=1e-6, atol=0) and torch.allclose(grad.cpu().sum(1), torch.zeros(6), atol=1e-7)


def test_refusals(tq):
    f = lambda *s: torch.ones(s, device="cuda")
    tok = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in ((f(3, 4, 5), tok), (f(3, 5), tok[:2])):
        with pytest.raises(ValueError):
            tq.tq_token_logp(*bad)
    with pytest.raises(TypeError):
        tq.tq_token_logp(f(3, 5), tok.float())
    with pytest.raises(TypeError):
        tq.tq_token_logp(f(3, 5).double(), tok)
    for args, kw in (((f(4),), {}), ((f(3).half(),), {}), ((f(3),), {"old_logp": f(2)}), ((f(3),), {"ref_logp": f(2)})):
        with pytest.raises(ValueError):
            tq.tq_policy_loss(f(3, 5), tok, *args, **kw)
    for kw in ({"clip_low": 1.5}, {"clip_low": -0.1}, {"clip_high": -1.0}, {"kl_coef": -1.0}, {"kl_coef": math.nan},
               {"temperature": 0.0}, {"clip_high": math.nan}):
        with pytest.raises(tq.TQError):
            tq.tq_policy_loss_grad(f(3, 5), tok, f(3), **kw)
    with pytest.raises(ValueError):
        tq.tq_policy_loss_backward(f(3, 5), tok, f(3), f(3), f(3, 3))
    with pytest.raises(ValueError):
        tq.tq_token_logp_backward(f(3, 5), tok, f(3, 2), f(2))
    with pytest.raises(ValueError):
        tq.tq_policy_loss_grad(f(3, 10)[:, ::2], tok, f(3), inplace=True)
