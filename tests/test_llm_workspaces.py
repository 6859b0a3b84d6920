"""Workspaces hold what their kernels write: the sizes against the partial rows
that each dispatch leaves (no GPU), and on the GPU exactly sized workspaces with
guard bytes on both sides, filled with NaN beforehand.  Refusals that rest on a
size are pinned to the check that makes them."""
import ctypes

import pytest
import torch

from gpu_util import note


@pytest.fixture(scope="module")
def tq():
    import tensor_quantization_amd as t
    return t


def cdiv(a, b):
    return -(-a // b)


def norm_parts(rows, cols, f32):
    """Rows of partial sums (dw and db each) of the norm's backward pass."""
    if cols < 8:                                        # 256 chunks of whole workgroups' rows
        return cdiv(rows, 256 * cdiv(cdiv(rows, 256), 256))
    if cols > (8192 if f32 else 16384):                 # 64 chunks of whole rounds of 16 rows
        return cdiv(rows, 16 * cdiv(cdiv(rows, 64), 16))
    teams = 512 // (64 if cols <= 512 else 128 if cols <= 1024 else 256 if cols <= 4096 else 512)
    return min(cdiv(rows, teams if cols <= 8192 else 1), 256)


@pytest.mark.parametrize("cols", [1, 7, 8, 512, 513, 1024, 1025, 2048, 4096, 8192, 8193, 16384, 16385, 40001])
@pytest.mark.parametrize("rows", [1, 3, 63, 64, 65, 255, 256, 257, 1000, 4097, 65536, 65537, 1 << 20])
def test_norm_backward(tq, rows, cols):
    have = tq.tq_layer_norm_backward_workspace_bytes(rows, cols)
    for f32 in (False, True):
        assert have >= norm_parts(rows, cols, f32) * 2 * cdiv(cols, 4) * 16


@pytest.mark.parametrize("N", [1, 7, 50, 512, 513, 11008, 1 << 23])
@pytest.mark.parametrize("M", [1, 64, 65, 80, 81, 100, 1000, 8192, 8193, 1 << 20])
def test_epilogue_backward(tq, M, N):
    have = tq.tq_linear_epilogue_backward_workspace_bytes(M, N)
    if M <= 64:
        assert have == 0                                # one chunk: its sums are dbias
        return
    chunk = 16 * cdiv(cdiv(M, max(1, 8192 // cdiv(N, 512))), 16)
    assert have >= cdiv(M, chunk) * cdiv(N, 4) * 16


@pytest.mark.parametrize("V", [1, 7, 4096, 4097, 8192, 8193, 32000, 131001, 131072, 1 << 20])
@pytest.mark.parametrize("rows", [1, 9, 127, 128, 511, 512, 2047, 2048, 5000])
@pytest.mark.parametrize("k", [1, 64, 1024])
def test_distillation(tq, rows, V, k):
    most = 8192 if rows * cdiv(V, 8192) >= 2048 else 4096
    parts = cdiv(V, 8 * cdiv(cdiv(V, cdiv(V, most)), 8))
    # a part's two pairs, and the logits at the entries
    assert tq.tq_topk_distill_workspace_bytes(rows, V, k) >= rows * (16 * parts + 4 * k)


def test_which_check_refuses(tq):
    P = ctypes.c_void_p
    A, B, C = P(0x10000), P(0x20000), P(0x30000)       # fake device addresses, never dereferenced
    n = tq.tq_topk_distill_workspace_bytes(1 << 30, 100, 5)

    def distill(rows, V, have):
        return tq._lib.tq_topk_distill_grad(A, 2, rows, V, V, A, 64, B, 0, 5, None, 1.0, None, C, B, V, A, have, None)
    assert distill(1 << 30, 100, n - 1) == tq.TQ_ERR_INVALID          # the workspace
    assert distill(1 << 31, 100, 1 << 62) == tq.TQ_ERR_UNSUPPORTED    # the rows
    assert distill(4, (1 << 31) - 255, 1 << 62) == tq.TQ_ERR_UNSUPPORTED
    for M in (65, 100, 8192):
        n = tq.tq_linear_epilogue_backward_workspace_bytes(M, 50)
        assert tq._lib.tq_linear_epilogue_backward(A, A, 2, M, 50, 1, B, C, A, n - 1, None) == tq.TQ_ERR_INVALID
    for rows, cols in ((300, 64), (300, 20001)):
        n = tq.tq_layer_norm_backward_workspace_bytes(rows, cols)
        assert tq._lib.tq_layer_norm_backward(A, A, 2, rows, cols, cols, cols, None, 0, C, C, A, B, B, A, n - 1,
                                              None) == tq.TQ_ERR_INVALID


# ------------------------------------------------------------------ on the GPU
GUARD = 4096


class Guarded:
    """n bytes between guards, all of them 0xff (NaNs) to begin with."""

    def __init__(self, n):
        self.n = n
        self.all = torch.full((GUARD + n + GUARD,), 255, dtype=torch.uint8, device="cuda")
        self.ptr = self.all.data_ptr() + GUARD

    def untouched(self):
        return bool((self.all[:GUARD] == 255).all()) and bool((self.all[GUARD + self.n:] == 255).all())


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 8), (70000, 7), (300, 500), (2100, 1000), (600, 4096), (300, 8192),
                                       (300, 16384), (1030, 16400), (65, 20001), (1, 40001)])
@pytest.mark.parametrize("ft", [torch.bfloat16, torch.float32])
def test_norm_backward_keeps_inside(tq, rows, cols, ft):
    note("norm backward, guarded workspace", rows, cols, ft)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn((rows, cols), generator=g, device="cuda").to(ft) for _ in range(2))
    _, mean, rstd = tq.tq_layer_norm(x)
    want = tq.tq_layer_norm_backward(dy, x, None, mean, rstd)
    ws = Guarded(tq.tq_layer_norm_backward_workspace_bytes(rows, cols))
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    assert 0 == tq._lib.tq_layer_norm_backward(dy.data_ptr(), x.data_ptr(), tq.FTYPE[ft], rows, cols, cols, cols, None,
                                               0, mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                                               db.data_ptr(), ws.ptr, ws.n, stream())
    assert ws.untouched() and all(torch.equal(a, b) for a, b in zip((dx, dw, db), want))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(64, 513), (65, 7), (65, 519), (100, 50), (8192, 520), (8192, 5), (8193, 1000)])
def test_epilogue_backward_keeps_inside(tq, M, N):
    note("epilogue backward, guarded workspace", M, N)
    g = torch.Generator(device="cuda").manual_seed(M)
    dy, z = (torch.randn((M, N), generator=g, device="cuda") for _ in range(2))
    want = tq.tq_linear_epilogue_backward(dy, z, "silu")
    ws = Guarded(tq.tq_linear_epilogue_backward_workspace_bytes(M, N))
    dz, db = torch.empty_like(dy), torch.empty(N, device="cuda")
    assert 0 == tq._lib.tq_linear_epilogue_backward(dy.data_ptr(), z.data_ptr(), 0, M, N, tq.ACT["silu"], dz.data_ptr(),
                                                    db.data_ptr(), ws.ptr if ws.n else None, ws.n, stream())
    assert ws.untouched() and torch.equal(dz, want[0]) and torch.equal(db, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,V,K", [(1, 5, 2), (3, 4097, 1024), (9, 131001, 32), (128, 70001, 64), (600, 33001, 5)])
@pytest.mark.parametrize("rest", [False, True])
def test_distillation_keeps_inside(tq, rows, V, K, rest):
    """Workspace, and the outputs that the backward pass is given: stats and
    rest_sum, a pair per row each."""
    note("distill, guarded workspace", rows, V, K, rest)
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((rows, V), generator=g, device="cuda")
    idx = (torch.arange(rows, device="cuda")[:, None] + 2 * torch.arange(K, device="cuda")[None]) % V
    val = torch.randn((rows, K), generator=g, device="cuda")
    tlse = torch.logsumexp(val, 1) + 0.5 if rest else None
    want_l, want_s, want_r = tq.tq_topk_distill(z, idx, val, teacher_lse=tlse)
    want_l2, want_g2 = tq.tq_topk_distill_grad(z, idx, val, teacher_lse=tlse)
    n = tq.tq_topk_distill_workspace_bytes(rows, V, K)
    head = (z.data_ptr(), 0, rows, V, V, idx.data_ptr(), 64, val.data_ptr(), 0, K, tlse.data_ptr() if rest else None, 1.0)
    ws, loss, stats, extra = Guarded(n), Guarded(4 * rows), Guarded(8 * rows), Guarded(8 * rows)
    assert 0 == tq._lib.tq_topk_distill(*head, loss.ptr, stats.ptr, extra.ptr, ws.ptr, n, stream())

    def floats(b):
        return b.all[GUARD:GUARD + b.n].view(torch.float32)
    assert all(b.untouched() for b in (ws, loss, stats, extra))
    assert torch.equal(floats(loss), want_l) and torch.equal(floats(stats).view(rows, 2), want_s)
    assert torch.equal(floats(extra).view(rows, 2), want_r) if rest else bool(torch.isnan(floats(extra)).all())
    ws, dz = Guarded(n), torch.empty_like(z)
    assert 0 == tq._lib.tq_topk_distill_grad(*head, None, loss.ptr, dz.data_ptr(), V, ws.ptr, n, stream())
    assert ws.untouched() and torch.equal(floats(loss), want_l2) and torch.equal(dz, want_g2)
