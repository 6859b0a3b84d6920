"""Host-side checks of the calls around a quantized layer (no GPU): malformed
arguments are refused before anything is enqueued, empty calls enqueue nothing,
and the workspaces have the sizes their kernels fill."""
import ctypes

import pytest

P = ctypes.c_void_p
A, B, C = P(0x10000), P(0x20000), P(0x30000)     # fake device addresses, never dereferenced
ODD2, ODD4, ODD8 = P(0x10001), P(0x10002), P(0x10004)
BIG = 1 << 40


@pytest.fixture(scope="module")
def tq():
    import tensor_quantization_amd as t
    return t


def test_layer_norm_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    f = L.tq_layer_norm
    assert f(None, 2, 4, 64, 64, B, B, 0, 1e-5, C, None, None, None) == INV
    assert f(A, 3, 4, 64, 64, B, B, 0, 1e-5, C, None, None, None) == INV          # x's type
    assert f(A, 2, 4, 64, 64, B, B, 9, 1e-5, C, None, None, None) == INV          # the parameters' type
    assert f(A, 2, -1, 64, 64, B, B, 0, 1e-5, C, None, None, None) == INV
    assert f(A, 2, 4, 64, 63, B, B, 0, 1e-5, C, None, None, None) == INV          # rows overlap
    assert f(A, 2, 4, 64, 64, B, B, 0, -1e-5, C, None, None, None) == INV
    assert f(A, 2, 4, 64, 64, B, B, 0, float("nan"), C, None, None, None) == INV
    assert f(A, 2, 4, 64, 64, B, B, 0, 1e-5, None, None, None, None) == INV       # no output
    assert f(A, 2, 1 << 31, 64, 64, B, B, 0, 1e-5, C, None, None, None) == UNS
    assert f(A, 2, 4, 1 << 31, 1 << 31, B, B, 0, 1e-5, C, None, None, None) == UNS
    assert f(ODD2, 2, 4, 64, 64, B, B, 0, 1e-5, C, None, None, None) == ALIGN
    assert f(ODD4, 0, 4, 64, 64, B, B, 0, 1e-5, C, None, None, None) == ALIGN
    assert f(A, 2, 4, 64, 64, ODD4, B, 0, 1e-5, C, None, None, None) == ALIGN     # f32 weight on 2 bytes
    assert f(A, 2, 4, 64, 64, B, B, 0, 1e-5, C, ODD4, None, None) == ALIGN        # mean
    assert f(A, 2, 0, 64, 64, B, B, 0, 1e-5, C, None, None, None) == 0
    assert f(None, 2, 4, 0, 0, None, None, 0, 1e-5, None, None, None, None) == 0
    q = L.tq_layer_norm_quant_per_token
    assert q(A, 2, 4, 64, 64, B, B, 0, 1e-5, None, C, None, None, None) == INV
    assert q(A, 2, 4, 64, 64, B, B, 0, 1e-5, C, None, None, None, None) == INV    # no scale
    assert q(A, 2, 4, 64, 64, B, B, 0, 1e-5, C, ODD4, None, None, None) == ALIGN
    g = L.tq_layer_norm_backward
    n = tq.tq_layer_norm_backward_workspace_bytes(4, 64)
    assert n >= 2 * 64 * 4
    assert g(A, A, 2, 4, 64, 64, 64, B, 0, C, C, A, B, B, None, n, None) == INV   # no workspace
    assert g(A, A, 2, 4, 64, 64, 64, B, 0, C, C, A, B, B, A, n - 1, None) == INV
    assert g(A, A, 2, 4, 64, 64, 64, B, 0, C, C, A, B, B, ODD8, n, None) == ALIGN
    assert g(None, A, 2, 4, 64, 64, 64, B, 0, C, C, A, B, B, A, n, None) == INV
    assert g(A, A, 2, 4, 64, 64, 64, B, 0, None, C, A, B, B, A, n, None) == INV   # no mean
    assert g(A, A, 2, 4, 64, 60, 64, B, 0, C, C, A, B, B, A, n, None) == INV      # dy's rows overlap
    assert g(A, A, 2, 4, 64, 64, 64, None, 7, C, C, A, B, None, A, n, None) == INV  # dweight's type
    assert g(A, A, 2, 4, 64, 64, 64, B, 0, C, C, None, None, None, None, 0, None) == 0   # nothing asked for


def test_epilogue_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    f = L.tq_w8a8_linear_epilogue
    ok = dict(qx=A, sx=B, qw=A, sw=B, M=4, N=8, K=16, bias=C, bdt=2, act=1, res=C, ldr=8, y=B, z=None, ydt=2, st=None)

    def call(**kw):
        return f(*{**ok, **kw}.values())
    assert call(qx=None) == INV and call(sx=None) == INV and call(sw=None) == INV and call(y=None) == INV
    assert call(act=5) == INV and call(act=-1) == INV
    assert call(ydt=4) == INV and call(bdt=4) == INV
    assert call(M=-1) == INV and call(ldr=7) == INV
    assert call(K=131072) == UNS and call(M=65535 * 128 + 1) == UNS
    assert call(sx=ODD4) == ALIGN and call(bias=ODD2) == ALIGN and call(res=ODD2) == ALIGN
    assert call(y=ODD2) == ALIGN and call(z=ODD4, ydt=0, bias=None, res=None) == ALIGN
    assert call(M=0) == 0 and call(N=0) == 0
    g = L.tq_linear_epilogue_backward
    n = tq.tq_linear_epilogue_backward_workspace_bytes(100, 50)
    assert n >= 50 * 4
    assert g(A, None, 2, 100, 50, 1, B, C, A, n, None) == INV
    assert g(A, A, 2, 100, 50, 7, B, C, A, n, None) == INV
    assert g(A, A, 5, 100, 50, 1, B, C, A, n, None) == INV
    assert g(A, A, 2, 100, 50, 1, None, C, A, n, None) == INV
    assert g(A, A, 2, 100, 50, 1, B, C, None, n, None) == INV
    assert g(A, A, 2, 100, 50, 1, B, C, A, n - 1, None) == INV
    assert g(A, A, 2, 100, 50, 1, B, C, ODD8, n, None) == ALIGN
    assert g(A, ODD2, 2, 100, 50, 1, B, C, A, n, None) == ALIGN
    assert g(A, A, 2, 100, 0, 1, B, C, A, 0, None) == 0


def test_distill_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    n = tq.tq_topk_distill_workspace_bytes(4, 100, 5)
    ok = dict(z=A, dt=2, rows=4, V=100, ld=100, idx=A, bits=64, val=B, vdt=0, k=5, tlse=None, T=1.0, dloss=None,
              loss=C, dz=B, ldd=100, ws=A, n=n, st=None)

    def call(**kw):
        return L.tq_topk_distill_grad(*{**ok, **kw}.values())
    assert call(z=None) == INV and call(idx=None) == INV and call(val=None) == INV and call(loss=None) == INV
    assert call(dt=3) == INV and call(vdt=3) == INV and call(bits=16) == INV
    assert call(k=0) == INV and call(rows=-1) == INV and call(V=0) == INV
    assert call(ld=99) == INV and call(ldd=99) == INV and call(dz=None) == INV
    for t in (0.0, -1.0, float("nan"), float("inf")):
        assert call(T=t) == INV
    assert call(ws=None) == INV and call(n=n - 1) == INV and call(ws=ODD8) == ALIGN
    assert call(k=1025) == UNS and call(V=1 << 31, ld=1 << 31, ldd=1 << 31) == UNS
    assert call(rows=1 << 30) == UNS or call(rows=1 << 30) == INV
    assert call(z=ODD2) == ALIGN and call(idx=ODD8) == ALIGN and call(val=ODD4) == ALIGN
    assert call(idx=ODD4, bits=32) == ALIGN and call(dloss=ODD4) == ALIGN
    assert call(rows=0) == 0
    f = L.tq_topk_distill
    assert f(A, 2, 4, 100, 100, A, 64, B, 0, 5, None, 1.0, None, None, None, A, n, None) == INV   # no loss
    b = L.tq_topk_distill_backward
    assert b(A, 2, 4, 100, 100, A, 64, B, 0, 5, None, 1.0, None, None, None, B, 100, None) == INV  # no stats
    assert b(A, 2, 4, 100, 100, A, 64, B, 0, 5, C, 1.0, C, None, None, B, 100, None) == INV        # no rest


def test_workspaces_grow_with_what_they_hold(tq):
    assert tq.tq_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert tq.tq_linear_epilogue_backward_workspace_bytes(64, 0) == 0
    assert tq.tq_topk_distill_workspace_bytes(0, 5, 5) == 0
    for rows in (1, 100, 10000):
        for cols in (1, 5, 4096, 40000):
            parts = tq.tq_layer_norm_backward_workspace_bytes(rows, cols) // 8
            assert parts >= (cols + 3) // 4 * 4 * min(rows, 1)
            assert tq.tq_topk_distill_workspace_bytes(rows, cols, 7) >= rows * 4 * 10
