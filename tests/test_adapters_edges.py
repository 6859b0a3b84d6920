"""GPU parity of the W8A8 product beside adapters at the edges of binary32: zeros
keep their sign for a token without an adapter."""
import pytest
import torch

import llm_util as ref
from test_parity_adapters import operands

pytestmark = pytest.mark.gpu


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
