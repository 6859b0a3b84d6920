"""GPU parity of distillation where a row's logits are far from zero or far
apart: common offsets, masks of large finite values, confident students.  The
loss depends on differences of logits alone, so the bounds are those of the
other parity tests.  Rows that a workgroup holds and rows in parts."""
import math

import pytest
import torch

import llm_util as ref
from gpu_util import note
from test_parity_distill import check, draw

pytestmark = pytest.mark.gpu

# (rows, columns, type): held by 256 threads, by 512, in parts
PATHS = [(7, 2000, "f32"), (130, 17001, "f32"), (7, 70001, "f32"), (7, 2000, "bf16"), (7, 2003, "f16"),
         (7, 70001, "f16")]


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("rows,V,ft", PATHS)
@pytest.mark.parametrize("T", [1.0, 0.3])
@pytest.mark.parametrize("rest", [False, True])
def test_common_offsets(tq, rows, V, ft, T, rest):
    """Rows whose logits share a large offset, and rows of one value that a
    program uses as a mask."""
    note("distill offsets", rows, V, ft, T, rest)
    z, idx, val, tlse, dloss = draw(rows, V, 12, V + 1, "f32")
    tlse = (torch.logsumexp(val.double() / T, 1) + 0.1).float()
    top = 6.0e4 if ft == "f16" else 1.0e5
    z[0] += 1.0e3
    z[1] += 1.0e4
    z[2] -= 3.0e4
    z[3] += top
    z[4] = -65504.0
    z[5] = -6.0e4 if ft == "f16" else -1.0e9
    check(tq, z.to(ref.TORCH[ft]), idx, val, T, tlse if rest else None, dloss, ft, "T %g" % T)
