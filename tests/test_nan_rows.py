"""GPU: a NaN is not lost on its way through the fused norm and quantizer, the
product and the slope of an activation, and stays in its row."""

import math

import pytest
import torch

import llm_util as ref
from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


# every variant: below one vector, by waves, by workgroups, longer than a workgroup holds
@pytest.mark.parametrize("cols", [5, 8, 300, 1000, 1500, 4096, 4099, 8000, 16000, 20001])
@pytest.mark.parametrize("ft", ["f32", "f16", "bf16"])
def test_fused_codes_of_a_nan(tq, cols, ft):
    note("nan through norm and quantizer", cols, ft)
    g = torch.Generator().manual_seed(cols)
    x = torch.randn((6, cols), generator=g)
    clean = x.to(ref.TORCH[ft]).cuda()
    x[1, cols - 1] = math.nan
    x[3, 0] = math.inf                       # its mean is infinite, its y NaN
    x = x.to(ref.TORCH[ft]).cuda()
    q, s, mean, rstd = tq.tq_layer_norm_quant_per_token(x, stats=True)
    q2, s2 = tq.tq_layer_norm_quant_per_token(clean)
    good, bad = [0, 2, 4, 5], [1, 3]
    assert torch.isnan(s[bad]).all() and torch.isnan(rstd[bad]).all()
    assert torch.equal(q[good], q2[good]) and torch.equal(s[good], s2[good])
    w = torch.ones(cols, device="cuda")
    w[cols // 2] = math.nan                  # a weight's NaN reaches every row
    assert torch.isnan(tq.tq_layer_norm_quant_per_token(x, w)[1]).all()
    # and what is computed from the codes
    qw = torch.randint(-127, 128, (40, cols), generator=g, dtype=torch.int64).to(torch.int8).cuda()
    y = tq.tq_w8a8_linear_epilogue(q, s, qw, torch.ones(40, device="cuda"), act="relu")
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[good]).all()


# one launch, chunks of rows, fewer than eight columns
@pytest.mark.parametrize("M,N", [(3, 24), (200, 520), (200, 5)])
@pytest.mark.parametrize("ft", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_slope_at_a_nan(tq, M, N, ft, act):
    note("nan through an activation's slope", M, N, ft, act)
    g = torch.Generator().manual_seed(M + N)
    dy, z = (torch.randn((M, N), generator=g).to(ref.TORCH[ft]).cuda() for _ in range(2))
    clean, _ = tq.tq_linear_epilogue_backward(dy, z, act)
    z[1, 2] = math.nan
    dz, db = tq.tq_linear_epilogue_backward(dy, z, act)
    at = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    at[1, 2] = act != "none"
    assert torch.isnan(dz[at]).all() and torch.equal(dz[~at], clean[~at])
    assert torch.equal(torch.isnan(db), at.any(0))
    z[1, 2], dy[1, 2] = 1.0, math.nan        # a gradient's NaN, where the slope is not 0
    dz, db = tq.tq_linear_epilogue_backward(dy, z, act)
    assert bool(torch.isnan(dz[1, 2])) and bool(torch.isnan(db[2]))
    z[1, 2] = -1.0
    dz, _ = tq.tq_linear_epilogue_backward(dy, z, act)
    assert bool(dz[1, 2] == 0) if act == "relu" else bool(torch.isnan(dz[1, 2]))
