"""GPU: tensors without rows or columns give outputs without rows, never
unwritten ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("shape", [(5, 0), (0, 5), (0, 0), (2, 3, 0), (2, 0, 3)])
def test_norm_without_elements(tq, shape):
    x = torch.empty(shape, device="cuda")
    y, mean, rstd = tq.tq_layer_norm(x)
    assert y.shape == x.shape and mean.shape == (0,) and rstd.shape == (0,)
    q, s = tq.tq_layer_norm_quant_per_token(x)
    assert q.shape == x.shape and s.shape == tq.tq_quant_per_token(y)[1].shape == (0,)
    dx, dw, db = tq.tq_layer_norm_backward(y, x, None, mean, rstd)
    assert dx.shape == x.shape and dw.shape == db.shape == shape[-1:]
    assert not dw.any() and not db.any()     # sums over no rows
