"""GPU parity of the products on codes either side of the rules that choose their
kernels: integer sums that binary32 holds are exact, so with scales of one every
output is; and epilogues at the sizes that only the tiles take."""
import pytest
import torch

from gpu_util import note
from test_parity_epilogue import ACTS, check as check_product, operands
from test_parity_gated import check as check_gated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    import tensor_quantization_amd as t
    return t


def exact(tq, M, N, K, offset=0):
    """K (127)^2 < 2^24: products, and both halves of the gated one, without a rounding."""
    assert K * 127 * 127 < 2 ** 24 and N % 2 == 0
    g = torch.Generator().manual_seed(M + N + K)
    qx, qw = (torch.randint(-127, 128, (r, K), generator=g, dtype=torch.int8) for r in (M, N))
    want = (qx.double() @ qw.double().T).float()

    def on_card(t):
        return torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape).copy_(t)
    one = [torch.ones(n, device="cuda") for n in (M, N, N // 2)]
    x, w = on_card(qx), on_card(qw)
    y = tq.tq_w8a8_linear_epilogue(x, one[0], w, one[1], out_dtype=torch.float32)
    assert torch.equal(y.cpu(), want)
    wg, wu = on_card(qw[:N // 2]), on_card(qw[N // 2:])
    _, z = tq.tq_w8a8_gated_linear(x, one[0], wg, one[2], wu, one[2], act="none", out_dtype=torch.float32, preact=True)
    assert torch.equal(z.cpu(), want)


# pieces of 32 x 16 and 32 x 32 up to and past 256, up to 16, 32 and 64 tokens, up to 6144 columns
@pytest.mark.parametrize("M,N", [(16, 8200), (17, 6144), (17, 6146), (32, 6144), (33, 4096), (32, 8192), (32, 8194),
                                 (33, 4098), (64, 2048), (64, 2050), (64, 4096), (64, 4098), (256, 512), (256, 514),
                                 (512, 256), (512, 512), (513, 512), (512, 514), (8192, 32), (8193, 32), (8192, 34)])
@pytest.mark.parametrize("K,offset", [(272, 0), (272, 8), (391, 0), (1030, 3)])
def test_either_side(tq, M, N, K, offset):
    note("product rules", M, N, K, offset)
    exact(tq, M, N, K, offset)


# the smallest tiles at any alignment: every number of whole blocks in flight
@pytest.mark.parametrize("K", [1, 15, 64, 127, 128, 129, 250, 257, 385, 513, 645, 770, 900, 1029, 1040])
def test_smallest_tiles(tq, K):
    exact(tq, 520, 1030, K, offset=1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("ft", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [131, 272, 514])
def test_smallest_tiles_epilogues(tq, K, ft, act):
    note("smallest tiles", K, ft, act)
    check_product(tq, 530, 541, K, ft, act, True, True)
    check_product(tq, 600, 500, K, ft, act, False, False)
    check_gated(tq, 530, 271, K, ft, act)
    check_gated(tq, 600, 250, K, ft, act, (False, True))


@pytest.mark.parametrize("K", [272, 275])
def test_smallest_tiles_strided_residual(tq, K):
    M, N = 600, 501
    qx, sx, qw, sw, bias, res = (t.cuda() for t in operands(M, N, K, 8))
    want = tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, bias=bias, residual=res)
    wide = torch.full((M, N + 7), float("nan"), dtype=res.dtype, device="cuda")
    wide[:, 3:3 + N] = res
    assert torch.equal(tq.tq_w8a8_linear_epilogue(qx, sx, qw, sw, bias=bias, residual=wide[:, 3:3 + N]), want)
