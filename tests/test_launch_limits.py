"""Sizes whose threads do not fit one launch (a grid holds fewer than 2^32 of
them): the calls around a quantized layer take them in several, or refuse them
before anything is enqueued."""
import ctypes

import pytest
import torch

import llm_util as ref
from gpu_util import note


@pytest.fixture(scope="module")
def tq():
    import tensor_quantization_amd as t
    return t


def test_products_beyond_a_grid_are_refused(tq):
    A, B = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)     # fake device addresses, never dereferenced
    f, g = tq._lib.tq_w8a8_linear_epilogue, tq._lib.tq_linear_epilogue_backward

    def product(M, N):
        return f(A, A, A, A, M, N, 16, None, 0, 0, None, N, B, None, 2, None)
    assert product(1, (1 << 27) - 15) == tq.TQ_ERR_UNSUPPORTED
    assert product(1 << 20, 1 << 26) == tq.TQ_ERR_UNSUPPORTED
    assert g(A, A, 2, 4, (1 << 33) - 511, 0, B, None, None, 0, None) == tq.TQ_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_norm_of_more_rows_than_a_grid_holds(tq):
    rows, cols = (1 << 26) + 5, 8
    note("norm", rows, cols)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w, b = 1 + 0.25 * torch.arange(cols, device="cuda"), 0.125 * torch.arange(cols, device="cuda")
    pick = [0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, 5 << 21, (1 << 26) - 1, 1 << 26, rows - 1]
    small, wc, bc = x[pick].cpu(), w.cpu(), b.cpu()
    y, mean, rstd = tq.tq_layer_norm(x, w, b)
    ty, tm, tr = ref.layer_norm_tol(small, wc, bc, 1e-5, "bf16")
    wy, wm, wr, _ = ref.layer_norm(small, wc, bc, 1e-5)
    ref.assert_within(y[pick], wy, ty, "y")
    ref.assert_within(mean[pick], wm[:, 0], tm[:, 0], "mean")
    ref.assert_within(rstd[pick], wr[:, 0], tr[:, 0], "rstd")
    q, s = tq.tq_layer_norm_quant_per_token(x, w, b)
    q2, s2, _ = tq.tq_quant_per_token(y[pick].contiguous())
    assert torch.equal(q[pick], q2) and torch.equal(s[pick], s2)
    dx, _, _ = tq.tq_layer_norm_backward(y, x, w, mean, rstd)
    args = (y[pick].cpu(), small, wc, mean[pick].cpu(), rstd[pick].cpu())
    ref.assert_within(dx[pick], ref.layer_norm_backward(*args)[0], ref.layer_norm_backward_tol(*args, "bf16", "f32")[0],
                      "dx")


@pytest.mark.gpu
def test_norm_backward_of_more_columns_than_a_grid_holds(tq):
    cols = (1 << 29) + 40
    note("norm backward", 1, cols)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    mean, rstd = torch.tensor([0.25], device="cuda"), torch.tensor([1.5], device="cuda")
    _, dw, db = tq.tq_layer_norm_backward(dy, x, None, mean, rstd)
    pick = [0, 1, (1 << 28) - 1, 1 << 28, (1 << 28) + 1, (1 << 29) - 1, 1 << 29, cols - 1]
    d = dy[0, pick].cpu().double()
    want = d * (x[0, pick].cpu().double() - 0.25) * 1.5          # one row: no sum, three roundings
    ref.assert_within(dw[pick], want, 4 * ref.U * want.abs(), "dw")
    ref.assert_within(db[pick], d, 0.0 * d, "db")


@pytest.mark.gpu
def test_distillation_of_more_rows_than_a_grid_holds(tq):
    rows, V, K = (1 << 24) + 3, 5, 2
    note("distill", rows, V, K)
    g = torch.Generator(device="cuda").manual_seed(7)
    z = torch.empty((rows, V), dtype=torch.float16, device="cuda").normal_(generator=g)
    val = torch.empty((rows, K), device="cuda").normal_(generator=g)
    idx = (torch.arange(rows, device="cuda", dtype=torch.int32)[:, None] + torch.tensor([0, 2], device="cuda")).int() % V
    tlse = torch.logsumexp(val, 1) + 0.25
    dloss = 0.5 + torch.rand(rows, generator=g, device="cuda")
    pick = [0, 1, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) - 1, 1 << 24, rows - 1]
    small = [t[pick].cpu() for t in (z, idx, val, tlse, dloss)]
    want, tol, want_l = ref.distill_grad(small[0].double(), small[1], small[2], 1.0, small[3], small[4])
    tol_l = ref.distill_loss_tol(small[0], small[1], small[2], 1.0, small[3])
    loss, stats, rest = tq.tq_topk_distill(z, idx, val, teacher_lse=tlse)
    grad = tq.tq_topk_distill_backward(z, idx, val, stats, dloss, teacher_lse=tlse, rest_sum=rest)
    loss2, grad2 = tq.tq_topk_distill_grad(z, idx, val, dloss=dloss, teacher_lse=tlse)
    for l, d in ((loss, grad), (loss2, grad2)):
        ref.assert_within(l[pick], want_l, tol_l, "loss")
        ref.assert_within(d[pick], want, tol + ref.rounding(want, "f16"), "gradient")
