"""GPU parity of the gate where its activation is almost nothing: far on the
negative side the value is compared relative to itself, which an absolute bound there
cannot."""
import pytest
import torch

import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu
U = ref.U

# the most negative gate at which value and slope are still normal numbers
FAR = {"silu": -82.0, "gelu": -12.5, "gelu_tanh": -9.5}


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def relative(g, act):
    """What act(g) and act'(g) may be off by, relative to themselves, at g <= -2.5.
    Each is an exponential of an argument x that binary32 knows to a few U |x| (x's
    rounding, its factor's, and for the tanh form's cubic two more), so it is off by
    that much relative to itself; 16 U more for the exponential, the quotient and the
    products.  silu: x = g.  gelu: erfc(y) falls as exp(-y^2), y = |g| / sqrt 2
    rounded twice: 2 y^2 2 U = 2 g^2 U (and as much in the slope's exp(-g^2 / 2)),
    erfcf itself within 16 U.  gelu_tanh: x = 1.6 |g| + 0.0714 |g|^3.  A slope adds
    two terms of opposite sign.  silu's are p and -|g| (1 - p) p, 1 to 2.31 or more at
    g <= -2.5: (2.31 + 1) / (2.31 - 1) < 8/3 of their sum; the others' are further apart."""
    x = g.abs()
    if act == "silu":
        e = 3 * U * x
    elif act == "gelu":
        e = 4 * U * x ** 2 + 16 * U
    else:
        e = 5 * U * (1.6 * x + 0.0714 * x ** 3)
    return e + 16 * U


@pytest.mark.parametrize("act", list(FAR))
@pytest.mark.parametrize("M,F", [(40, 1000), (300, 7)])
def test_negative_tail(tq, act, M, F):
    note("gate tail", act, M, F)
    gen = torch.Generator().manual_seed(F)
    lo = FAR[act]
    gate = lo + (-2.5 - lo) * torch.rand((M, F), generator=gen)
    up, dy = (0.5 + torch.rand((M, F), generator=gen) for _ in range(2))
    z = torch.cat([gate, up], 1)
    g, u, d = gate.double(), up.double(), dy.double()
    a, s = ref.act(g, act), ref.act_slope(g, act)
    rel = relative(g, act)
    tiny = 2.0 ** -126                                  # a result that is no normal number may be 0
    ref.assert_within(tq.tq_gated_act(z.cuda(), act), a * u, (rel + 2 * U) * (a * u).abs() + tiny, "y")
    dz, db = tq.tq_gated_act_backward(dy.cuda(), z.cuda(), act)
    ref.assert_within(dz[:, F:], a * d, (rel + 2 * U) * (a * d).abs() + tiny, "du")
    ref.assert_within(dz[:, :F], d * u * s, (8 / 3 * rel + 4 * U) * (d * u * s).abs() + tiny, "dg")
    # far below any absolute bound, and not nothing
    assert bool((dz[:, F:][gate.cuda() > lo + 1] < 0).all())


@pytest.mark.parametrize("act", list(FAR))
@pytest.mark.parametrize("M,F", [(1, 64), (20, 40), (130, 96), (700, 520)])
def test_negative_tail_of_the_block(tq, act, M, F):
    """The block's gates are its biases (codes of 0): the same values from its epilogues."""
    gen = torch.Generator().manual_seed(M)
    K, lo = 144, FAR[act]
    qx, qu = (torch.randint(-127, 128, (n, K), generator=gen).to(torch.int8) for n in (M, F))
    bias = lo + (-2.5 - lo) * torch.rand(F, generator=gen)
    one = torch.ones(M), torch.zeros((F, K), dtype=torch.int8), torch.ones(F)
    # u = 1 exactly: no codes, a bias of 1
    args = [t.cuda() for t in (qx, one[0], one[1], one[2], 0 * qu, one[2])]
    y = tq.tq_w8a8_gated_linear(*args, bias_gate=bias.cuda(), bias_up=torch.ones(F).cuda(), act=act,
                                out_dtype=torch.float32)
    a = ref.act(bias.double(), act).expand(M, F)
    ref.assert_within(y, a, (relative(bias.double(), act) + 2 * U) * a.abs() + 2.0 ** -126, "y")
