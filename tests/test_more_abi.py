"""Host-side checks (no GPU) of the gated block's, the adapters' and the policy
loss's calls: malformed arguments are refused before anything is enqueued, empty
calls enqueue nothing, and the workspaces have the sizes their kernels fill."""
import ctypes

import pytest

P = ctypes.c_void_p
A, B, C = P(0x10000), P(0x20000), P(0x30000)     # fake device addresses, never dereferenced
ODD2, ODD4, ODD8 = P(0x10001), P(0x10002), P(0x10004)


@pytest.fixture(scope="module")
def tq():
    import tensor_quantization_amd as t
    return t


def cdiv(a, b):
    return -(-a // b)


def test_gated_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    ok = dict(qx=A, sx=B, qg=A, sg=B, qu=A, su=B, M=4, F=8, K=16, bg=C, bu=C, bdt=2, act=2, y=B, z=None, ydt=2, st=None)

    def call(**kw):
        return L.tq_w8a8_gated_linear(*{**ok, **kw}.values())
    for name in ("qx", "sx", "qg", "sg", "qu", "su", "y"):
        assert call(**{name: None}) == INV, name
    assert call(act=5) == INV and call(act=-1) == INV and call(ydt=3) == INV and call(bdt=3) == INV
    assert call(M=-1) == INV and call(F=-1) == INV and call(K=-1) == INV
    assert call(K=131072) == UNS and call(M=65535 * 128 + 1) == UNS and call(F=1 << 27) == UNS
    assert call(M=65535 * 128, F=1 << 20) == UNS                  # too many tiles
    for name in ("sx", "sg", "su"):
        assert call(**{name: ODD4}) == ALIGN, name
    assert call(bg=ODD2) == ALIGN and call(bu=ODD2) == ALIGN and call(y=ODD2) == ALIGN and call(z=ODD2) == ALIGN
    assert call(y=ODD4, ydt=0) == ALIGN
    assert call(M=0) == 0 and call(F=0) == 0
    f = L.tq_gated_act
    assert f(None, 2, 4, 8, 2, B, None) == INV and f(A, 2, 4, 8, 2, None, None) == INV
    assert f(A, 3, 4, 8, 2, B, None) == INV and f(A, 2, 4, 8, 9, B, None) == INV and f(A, 2, -4, 8, 2, B, None) == INV
    assert f(A, 2, 4, 1 << 31, 2, B, None) == UNS and f(ODD2, 2, 4, 8, 2, B, None) == ALIGN
    assert f(A, 2, 0, 8, 2, B, None) == 0 and f(None, 2, 4, 0, 2, None, None) == 0
    g = L.tq_gated_act_backward
    n = tq.tq_gated_act_backward_workspace_bytes(100, 50)
    assert n >= 100 * 4
    assert g(A, None, 2, 100, 50, 1, B, C, A, n, None) == INV and g(None, A, 2, 100, 50, 1, B, C, A, n, None) == INV
    assert g(A, A, 2, 100, 50, 7, B, C, A, n, None) == INV and g(A, A, 5, 100, 50, 1, B, C, A, n, None) == INV
    assert g(A, A, 2, 100, 50, 1, None, C, A, n, None) == INV and g(A, A, 2, 100, 50, 1, B, C, None, n, None) == INV
    assert g(A, A, 2, 100, 50, 1, B, C, A, n - 1, None) == INV
    assert g(A, A, 2, 100, 50, 1, B, C, ODD8, n, None) == ALIGN and g(A, ODD2, 2, 100, 50, 1, B, C, A, n, None) == ALIGN
    assert g(A, A, 2, 100, 50, 1, B, ODD4, A, n, None) == ALIGN
    assert g(A, A, 2, 100, 1 << 31, 1, B, C, A, 1 << 62, None) == UNS
    assert g(A, A, 2, 100, 0, 1, B, C, A, 0, None) == 0


@pytest.mark.parametrize("F", [1, 7, 50, 512, 513, 11008, 1 << 23])
@pytest.mark.parametrize("M", [1, 64, 65, 72, 73, 100, 1000, 8192, 8193, 1 << 20])
def test_gate_backward_workspace(tq, M, F):
    have = tq.tq_gated_act_backward_workspace_bytes(M, F)
    if M <= 64:
        assert have == 0                                # one chunk: its sums are dbias
        return
    chunk = 8 * cdiv(cdiv(M, max(1, 8192 // cdiv(F, 512))), 8)
    assert have >= cdiv(M, chunk) * cdiv(2 * F, 4) * 16


def test_adapter_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    n = tq.tq_w8a8_linear_adapters_workspace_bytes(4, 12)
    assert n >= 4 * 12 * 4 and tq.tq_w8a8_linear_adapters_workspace_bytes(0, 12) == 0
    ok = dict(x=A, xdt=2, ldx=16, qx=A, sx=B, qw=A, sw=B, M=4, N=8, K=16, ids=C, count=3, R=12, a=A, b=B, scale=C, bias=C,
              bdt=2, act=1, res=C, ldr=8, y=B, z=None, ydt=2, ws=A, n=n, st=None)

    def call(**kw):
        return L.tq_w8a8_linear_adapters(*{**ok, **kw}.values())
    for name in ("x", "qx", "sx", "qw", "sw", "ids", "a", "b", "y", "ws"):
        assert call(**{name: None}) == INV, name
    assert call(xdt=3) == INV and call(ydt=3) == INV and call(bdt=3) == INV and call(act=5) == INV
    assert call(M=-1) == INV and call(count=-1) == INV and call(R=0) == INV
    assert call(ldx=15) == INV and call(ldr=7) == INV and call(n=n - 1) == INV
    big = 1 << 62
    assert call(R=257, n=big) == UNS and call(K=131072, ldx=131072) == UNS and call(M=65535 * 128 + 1, n=big) == UNS
    assert call(count=1 << 31) == UNS
    for name in ("x", "a", "b", "bias", "res", "y", "z"):
        assert call(**{name: ODD2}) == ALIGN, name
    for name in ("sx", "sw", "ids", "scale"):
        assert call(**{name: ODD4}) == ALIGN, name
    assert call(ws=ODD8) == ALIGN
    assert call(M=0) == 0 and call(N=0) == 0


def test_policy_refusals(tq):
    L, INV, UNS, ALIGN = tq._lib, tq.TQ_ERR_INVALID, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_ALIGN
    V = 10000
    n = tq.tq_policy_loss_workspace_bytes(4, V)
    ok = dict(z=A, dt=2, rows=4, V=V, ld=V, tok=A, bits=64, adv=C, old=None, ref=None, lo=0.2, hi=0.2, beta=0.0, T=1.0,
              dloss=None, loss=C, logp=C, dz=B, ldd=V, ws=A, n=n, st=None)

    def call(**kw):
        return L.tq_policy_loss_grad(*{**ok, **kw}.values())
    for name in ("z", "tok", "adv", "loss", "logp", "dz", "ws"):
        assert call(**{name: None}) == INV, name
    assert call(dt=3) == INV and call(bits=16) == INV and call(rows=-1) == INV and call(V=0) == INV
    assert call(ld=V - 1) == INV and call(ldd=V - 1) == INV and call(n=n - 1) == INV
    for t in (0.0, -1.0, float("nan"), float("inf")):
        assert call(T=t) == INV
    for kw in ({"lo": -0.1}, {"lo": 1.1}, {"hi": -0.1}, {"beta": -1.0}, {"beta": float("inf")}, {"lo": float("nan")}):
        assert call(**kw) == INV and call(rows=0, **kw) == INV
    big = 1 << 62
    assert call(V=1 << 31, ld=1 << 31, ldd=1 << 31, n=big) == UNS and call(rows=1 << 31, n=big) == UNS
    assert call(z=ODD2) == ALIGN and call(tok=ODD8) == ALIGN and call(tok=ODD4, bits=32) == ALIGN and call(dz=ODD2) == ALIGN
    for name in ("adv", "old", "ref", "dloss", "loss", "logp"):
        assert call(**{name: ODD4}) == ALIGN, name
    assert call(ws=ODD8) == ALIGN and call(rows=0) == 0
    f = L.tq_token_logp
    assert f(A, 2, 4, V, V, A, 64, 1.0, None, None, A, n, None) == INV               # no output
    assert f(A, 2, 4, V, V, A, 64, 1.0, C, ODD4, A, n, None) == ALIGN
    assert f(A, 2, 4, V, V, A, 64, 1.0, C, None, A, n - 1, None) == INV
    b = L.tq_token_logp_backward
    assert b(A, 2, 4, V, V, A, 64, 1.0, None, None, B, V, None) == INV             # no stats
    assert b(A, 2, 4, V, V, A, 64, 1.0, C, None, B, V - 1, None) == INV
    g = L.tq_policy_loss_backward
    assert g(A, 2, 4, V, V, A, 64, C, None, None, 0.2, 0.2, 0.0, 1.0, None, C, None, B, V, None) == INV   # no logp
    assert g(A, 2, 4, V, V, A, 64, C, None, None, 0.2, 0.2, 0.0, 1.0, C, None, None, B, V, None) == INV   # no stats


@pytest.mark.parametrize("V", [1, 7, 4096, 4097, 8192, 8193, 32000, 131001, 131072, 1 << 20])
@pytest.mark.parametrize("rows", [1, 9, 127, 128, 511, 512, 2047, 2048, 5000])
def test_policy_workspace(tq, rows, V):
    if 8 <= V <= 8192:
        assert tq.tq_policy_loss_workspace_bytes(rows, V) == 0      # a workgroup per row, forwards and in one call
        return
    most = 8192 if rows * cdiv(V, 8192) >= 2048 else 4096
    parts = cdiv(V, 8 * cdiv(cdiv(V, cdiv(V, most)), 8))
    assert tq.tq_policy_loss_workspace_bytes(rows, V) >= rows * (8 * parts + 4)   # a part's pair, the token's logit
