"""GPU parity of the W8A8 product beside adapters at the edges of binary32: zeros
keep their sign for a token without an adapter, and what is infinite in an adapter
reaches its own tokens as the definition says, by every kernel."""
import math

import pytest
import torch

import llm_util as ref
from gpu_util import note
from test_parity_adapters import definition, operands

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def bits(t):
    return t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)


@pytest.mark.parametrize("M", [1, 12, 40, 130, 300, 700])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_zeros_keep_their_sign_without_an_adapter(tq, M, out):
    N, K, R, count = 300 if M < 700 else 900, 272, 16, 3
    ops = list(operands(M, N, K, R, count, M, "bf16", out))
    ops[1][::3] = 0                                     # sums of 0 ...
    ops[4][::2] *= -1                                   # ... times a negative scale: -0
    ops[5][:(M + 1) // 2] = -1
    dev = [t.cuda() for t in ops]
    none = dev[5] < 0
    for bias in (None, torch.full_like(dev[9], -0.0)):
        y, z = tq.tq_w8a8_linear_adapters(*dev[:8], scale=dev[8], bias=bias, act="none",
                                          out_dtype=ref.TORCH[out], preact=True)
        wy, wz = tq.tq_w8a8_linear_epilogue(*dev[1:5], bias=bias, act="none", out_dtype=ref.TORCH[out], preact=True)
        assert bool((wy[0] == 0).all()) and bool(torch.signbit(wy[0]).any())
        assert torch.equal(bits(y[none]), bits(wy[none])) and torch.equal(bits(z[none]), bits(wz[none]))


def few_and_tiles(M):
    return (136 if M < 600 else 1040), 272, 40, 4


# the few-token kernel and every tile
@pytest.mark.parametrize("M", [3, 40, 130, 300, 700, 2100, 4100])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [272, 269])
def test_infinities_in_b(tq, M, ft, K):
    """h of the ranks in question is far from 0 and of known sign: a sum with one
    infinite term is that infinity, one with two opposite ones is NaN."""
    note("adapters, infinite b", M, ft, K)
    N, _, R, count = few_and_tiles(M)
    if M > 700:
        N = M + 10
    ops = list(operands(M, N, K, R, count, M + K, ft, "f32"))
    ops[0], ops[5] = ops[0].abs(), torch.arange(M, dtype=torch.int32) % count
    a, b = ops[6], ops[7]
    for r, sign in ((0, 1), (7, -1), (33, 1), (39, -1)):
        a[:, r] = sign * a[:, r].abs()
    b[0, 5, 0] = INF
    b[0, 6, 7] = INF
    b[0, 70, 33] = -INF
    b[1, 5, 39] = INF
    b[1, 131, 33] = b[1, 131, 7] = INF                   # opposite terms
    b[2, 9, 0] = b[2, 9, 33] = -INF                     # like ones
    b[2, 10, 7] = math.nan
    dev = [t.cuda() for t in ops]
    y, z = tq.tq_w8a8_linear_adapters(*dev[:8], scale=dev[8], bias=dev[9], residual=dev[10], out_dtype=torch.float32,
                                      preact=True)
    wz, wy, tz, ty = definition(*ops, "none", ft, "f32")
    assert bool(torch.isinf(wz).any()) and bool(torch.isnan(wz).any())
    ref.assert_within(z, wz, tz, "z")
    ref.assert_within(y, wy, ty, "y")


@pytest.mark.parametrize("M", [3, 40, 300, 700])
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
def test_a_large_h_beside_an_infinite_one(tq, M, ft):
    """A rank of a is infinite, another one's h is finite but beyond f16's range and
    against it: the infinity stands."""
    N, K, R, count = few_and_tiles(M)
    ops = list(operands(M, N, K, R, count, M, ft, "f32"))
    ops[0], ops[5] = 1 + ops[0].abs(), torch.arange(M, dtype=torch.int32) % count
    a, b = ops[6], ops[7]
    a[1] = a[1].abs() + 1
    a[1, 3] = 300.0                                      # h = 300 K times x of at least 1: above 81600
    a[1, 2, 11] = INF
    b[1] = b[1].abs() + 0.25
    b[1, :, 3] *= -1
    dev = [t.cuda() for t in ops]
    y = tq.tq_w8a8_linear_adapters(*dev[:8], scale=dev[8], out_dtype=torch.float32)
    mine = dev[5] == 1
    assert bool((y[mine] == INF).all()), y[mine]
    assert bool(torch.isfinite(y[~mine]).all())
