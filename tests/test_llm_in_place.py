"""GPU: the epilogue's outputs over its inputs, as the header allows: dz over dy
or preact, y over the residual; the bits are those of separate buffers."""
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


def normal(shape, ft, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(ref.TORCH[ft]).cuda()


# one chunk and several; widths whose last vector is moved back, whose last slab is short, below one vector
@pytest.mark.parametrize("M", [1, 3, 64, 65, 300])
@pytest.mark.parametrize("N", [5, 8, 13, 512, 513, 519, 1030])
@pytest.mark.parametrize("act,ft", [("none", "bf16"), ("relu", "f32"), ("silu", "f16"), ("gelu", "f32"),
                                    ("gelu_tanh", "bf16")])
def test_dz_over_dy_or_preact(tq, M, N, act, ft):
    note("epilogue backward in place", M, N, act, ft)
    dy, z = normal((M, N), ft, M + N), normal((M, N), ft, M * N)
    want, want_db = tq.tq_linear_epilogue_backward(dy, z, act)
    n = tq.tq_linear_epilogue_backward_workspace_bytes(M, N)
    for over in (0, 1):
        a, b, db = dy.clone(), z.clone(), torch.empty(N, device="cuda")
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        out = (a, b)[over]
        s = tq._lib.tq_linear_epilogue_backward(a.data_ptr(), b.data_ptr(), tq.FTYPE[a.dtype], M, N, tq.ACT[act],
                                                out.data_ptr(), db.data_ptr(), ws.data_ptr(), n,
                                                torch.cuda.current_stream().cuda_stream)
        assert s == 0 and torch.equal(out, want) and torch.equal(db, want_db)


# a few tokens, small outputs, 64, 128 and 256 tiles, and operands of other alignments
@pytest.mark.parametrize("M,N,K", [(1, 130, 256), (30, 200, 272), (200, 1000, 400), (600, 1100, 272),
                                   (1500, 1600, 272), (4100, 4110, 144), (100, 130, 129), (1500, 1600, 133),
                                   (3000, 4110, 131)])
@pytest.mark.parametrize("ft,act", [("bf16", "silu"), ("f32", "none"), ("f16", "gelu_tanh")])
def test_y_over_the_residual(tq, M, N, K, ft, act):
    note("product in place", M, N, K, ft, act)
    g = torch.Generator(device="cuda").manual_seed(M + K)
    qx, qw = (torch.randint(-127, 128, s, generator=g, device="cuda").to(torch.int8) for s in ((M, K), (N, K)))
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda") / (80 * K)
    res = normal((M, N), ft, 3)
    want, want_z = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, act=act, residual=res, out_dtype=res.dtype, preact=True)
    for z in (None, torch.empty_like(res)):
        y = res.clone()
        s = tq._lib.tq_w8a8_linear_epilogue(qx.data_ptr(), sx.data_ptr(), qw.data_ptr(), sw.data_ptr(), M, N, K, None, 0,
                                            tq.ACT[act], y.data_ptr(), N, y.data_ptr(),
                                            None if z is None else z.data_ptr(), tq.FTYPE[y.dtype],
                                            torch.cuda.current_stream().cuda_stream)
        assert s == 0 and torch.equal(y, want)
        assert z is None or torch.equal(z, want_z)
