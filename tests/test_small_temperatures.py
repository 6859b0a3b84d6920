"""Host-side checks (no GPU): a temperature whose inverse overflows binary32 is refused
before anything is enqueued (every logit's difference times infinity would be NaN or
infinite)."""
import ctypes

import pytest

P = ctypes.c_void_p
A, B = P(0x10000), P(0x20000)                   # fake device addresses, never dereferenced
SMALL = (0.0, 1e-45, 1e-40, 2.9e-39, 9e-39)


@pytest.fixture(scope="module")
def tq():
    import tensor_quantization_amd as t
    return t


@pytest.mark.parametrize("T", SMALL)
def test_policy_loss(tq, T):
    L, INV = tq._lib, tq.TQ_ERR_INVALID
    head, policy = (A, 0, 4, 100, 100, B, 64), (B, None, None, 0.2, 0.2, 0.0)
    assert L.tq_token_logp(*head, T, B, None, None, 0, None) == INV
    assert L.tq_token_logp_backward(*head, T, B, None, A, 100, None) == INV
    assert L.tq_policy_loss(*head, *policy, T, B, B, None, None, 0, None) == INV
    assert L.tq_policy_loss_backward(*head, *policy, T, B, B, None, A, 100, None) == INV
    assert L.tq_policy_loss_grad(*head, *policy, T, None, B, B, A, 100, None, 0, None) == INV
    # just above the limit it is taken (no rows: nothing is enqueued)
    assert L.tq_token_logp(A, 0, 0, 100, 100, B, 64, 1.01e-38, None, None, None, 0, None) == 0


@pytest.mark.parametrize("T", SMALL)
def test_distillation(tq, T):
    L, INV = tq._lib, tq.TQ_ERR_INVALID
    head = (A, 0, 4, 100, 100, B, 64, B, 0, 8, None)
    assert L.tq_topk_distill(*head, T, B, B, None, A, 1 << 20, None) == INV
    assert L.tq_topk_distill_backward(*head, T, B, None, None, A, 100, None) == INV
    assert L.tq_topk_distill_grad(*head, T, None, B, A, 100, A, 1 << 20, None) == INV
    assert L.tq_topk_distill(A, 0, 0, 100, 100, B, 64, B, 0, 8, None, 1.01e-38, B, B, None, A, 1 << 20, None) == 0
