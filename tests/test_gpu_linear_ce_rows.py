"""The output head's loss where rows are masked, certain or very many: what must not enter its gradients, and
what is lost where p - 1 cancels or a sum is long."""
import pytest
import torch

from tests.test_gpu_linear_ce import IGNORE, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,V", [(5, 72, 300), (16, 264, 1000), (20, 64, 300), (140, 520, 700), (1000, 256, 2049)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_ignored_rows_of_hidden_states_may_hold_anything(rfq, T, D, V, bad):
    """A row that is ignored gives no gradient, whatever its hidden state holds (padding that was never written)."""
    h, w, labels, dloss = make(T, D, V, seed=T, ignore_share=0.3)
    labels[T - 1] = IGNORE
    masked = labels == IGNORE
    h[masked] = 0
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    want = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    h[masked] = bad
    loss, lse2 = rfq.linear_ce_alloc(h, w, labels)
    assert torch.equal(lse2[~masked], lse[~masked]) and not loss[masked].any()
    got = rfq.linear_ce_backward_alloc(h, w, labels, lse2, dloss)
    assert torch.equal(got[0], want[0]) and not got[0][masked].any()
    assert torch.equal(got[1], want[1])
    _, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse2, dloss, want_dh=False)
    assert torch.equal(dw, want[1])
