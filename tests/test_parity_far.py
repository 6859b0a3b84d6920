"""GPU parity of the gated block, the adapters and the policy loss where offsets
pass 32 bits: the last rows of tensors of more than 2^31 elements, and rows that
lie that far apart, have the bits of the same rows by themselves."""
import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 24


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def far_rows(t):
    """t's rows FAR elements apart."""
    wide = torch.empty((t.shape[0] - 1) * FAR + t.shape[1], dtype=t.dtype, device="cuda")
    v = wide.as_strided(t.shape, (FAR, 1))
    v.copy_(t)
    return v


def codes(g, *s):
    return torch.randint(-127, 128, s, generator=g, dtype=torch.int8).cuda()


@pytest.mark.parametrize("rows,V", [(3, 5), (3, 8200), (3, 140001)])
def test_logits(tq, rows, V):
    note("far logits", rows, V)
    g = torch.Generator().manual_seed(V)
    z = torch.randn((rows, V), generator=g).to(torch.bfloat16).cuda()
    token, adv = torch.tensor([V - 1, 0, V // 2]).cuda(), torch.tensor([1.0, -2.0, 0.5]).cuda()
    far = far_rows(z)
    want, got = (tq.tq_policy_loss_grad(t, token, adv, kl_coef=0.0) for t in (z, far))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    (wl, wlogp, wstats), (loss, logp, stats) = (tq.tq_policy_loss(t, token, adv) for t in (z, far))
    assert torch.equal(wl, loss) and torch.equal(wlogp, logp) and torch.equal(wstats, stats)
    assert torch.equal(tq.tq_policy_loss_backward(far, token, adv, logp, stats),
                       tq.tq_policy_loss_backward(z, token, adv, logp, stats))


def test_many_rows_held(tq):
    V, rows = 32000, 68000                             # 2.18e9 elements
    note("far logits", rows, V)
    z = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    z[-300:] = torch.randn((300, V), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    token = torch.arange(rows, device="cuda") % V
    adv = torch.ones(rows, device="cuda")
    loss, logp, dz = tq.tq_policy_loss_grad(z, token, adv)
    wl, wlogp, wdz = tq.tq_policy_loss_grad(z[-300:], token[-300:], adv[-300:])
    assert torch.equal(logp[-300:], wlogp) and torch.equal(loss[-300:], wl) and torch.equal(dz[-300:], wdz)
    l, stats = tq.tq_token_logp(z, token)
    wl, wstats = tq.tq_token_logp(z[-300:], token[-300:])
    assert torch.equal(l[-300:], wl) and torch.equal(stats[-300:], wstats)
    del dz
    d = tq.tq_token_logp_backward(z, token, stats)
    assert torch.equal(d[-300:], tq.tq_token_logp_backward(z[-300:], token[-300:], wstats))


def test_gate(tq):
    M, F = 66000, 16392                                # 2.16e9 elements of z
    note("far gate", M, F)
    g = torch.Generator().manual_seed(2)
    z = torch.zeros((M, 2 * F), dtype=torch.bfloat16, device="cuda")
    tail, dy = torch.randn((9, 2 * F), generator=g).to(torch.bfloat16).cuda(), torch.ones((M, F), dtype=torch.bfloat16,
                                                                                         device="cuda")
    z[-9:] = tail
    y = tq.tq_gated_act(z, "silu")
    assert torch.equal(y[-9:], tq.tq_gated_act(tail, "silu")) and not bool(y[:9].any())
    del y
    dz, db = tq.tq_gated_act_backward(dy, z, "silu")
    wz, wb = tq.tq_gated_act_backward(dy[-9:], tail, "silu")
    assert torch.equal(dz[-9:], wz)
    # rows of zeros add nothing; nine rows' sums in another order
    assert torch.allclose(db, wb, rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("K", [64, 67])
def test_products(tq, K):
    M, F = 66000, 16392                                # 2.16e9 elements of the kept values and of the adapters' output
    note("far products", M, F, K)
    g = torch.Generator().manual_seed(K)
    q = codes(g, M, K)
    s = torch.rand(M, generator=g).cuda()
    w = codes(g, 2 * F, K)
    sw = torch.rand(2 * F, generator=g).cuda()
    y, z = tq.tq_w8a8_gated_linear(q, s, w[:F], sw[:F], w[F:], sw[F:], preact=True)
    wy, wz = tq.tq_w8a8_gated_linear(q[-300:], s[-300:], w[:F], sw[:F], w[F:], sw[F:], preact=True)
    assert torch.equal(y[-300:], wy) and torch.equal(z[-300:], wz)
    del y, z
    R = 8
    x = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
    a, b = (torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((3, R, K), (3, 2 * F, R)))
    ids = (torch.arange(M, dtype=torch.int32) % 4).cuda()
    y = tq.tq_w8a8_linear_adapters(x, q, s, w, sw, ids, a, b)
    want = tq.tq_w8a8_linear_adapters(x[-1200:], q[-1200:], s[-1200:], w, sw, ids[-1200:], a, b)
    assert torch.equal(y[-1200:], want)


def test_strided_x_of_adapters(tq):
    g = torch.Generator().manual_seed(3)
    M, N, K, R = 3, 100, 300, 16
    x = torch.randn((M, K), generator=g).to(torch.bfloat16).cuda()
    q, w, ids = codes(g, M, K), codes(g, N, K), torch.tensor([1, 2, 0], dtype=torch.int32).cuda()
    s, sw = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    a, b = (torch.randn(v, generator=g).to(torch.bfloat16).cuda() for v in ((2, R, K), (2, N, R)))
    assert torch.equal(tq.tq_w8a8_linear_adapters(far_rows(x), q, s, w, sw, ids, a, b),
                       tq.tq_w8a8_linear_adapters(x, q, s, w, sw, ids, a, b))
