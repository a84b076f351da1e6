"""Failure detection at the output head without a GPU fault: every wait in its products is bounded, and a wait that
runs out leaves a usable context.

The library's test hook leaves out the last stage fill of the first CTA's only tile, so its MMA warp waits for
that stage until the limit (about 1.5 s) and raises the CTA's abort flag; the epilogue's warps, of which the last
holds rows past the end of h here, learn of it at a wait of their own and give up together.  In a pair the other CTA's
epilogue runs into its own limit, twice as long.  The calls that follow are right to the last bit.
"""
import pytest
import torch

from tests.test_gpu_linear_ce import make

pytestmark = pytest.mark.gpu

D = 1024


# one CTA a tile of 64 columns, one a tile of 256, CTA pairs
@pytest.mark.parametrize("T,V", [(100, 300), (100, 20000), (300, 300)])
@pytest.mark.parametrize("backward", [False, True])
def test_skipped_fill_times_out_and_the_next_call_is_right(rfq, T, V, backward):
    h, w, labels, dloss = make(T, D, V, seed=T)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    torch.cuda.synchronize()
    rfq.check_device_error()

    rfq.debug_skip_next_fill(D // 64 - 1)
    if backward:
        rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    else:
        rfq.linear_ce_alloc(h, w, labels)
    with pytest.raises(rfq.RFQError) as info:
        rfq.check_device_error()
    assert info.value.status == 6          # RFQ_ERR_TIMEOUT
    assert info.value.detail == 1          # the MMA warp's wait for a loaded stage
    rfq.check_device_error()               # the error word was cleared

    again = rfq.linear_ce_alloc(h, w, labels)
    grads = rfq.linear_ce_backward_alloc(h, w, labels, again[1], dloss)
    torch.cuda.synchronize()
    rfq.check_device_error()
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dh, dw), again + grads))


@pytest.mark.parametrize("T", [1, 31, 33, 97, 127, 129, 161, 255, 257, 383])
def test_rows_that_end_inside_a_warp(rfq, T):
    """Lanes past the last row leave the epilogue's loop early and come together again: many tiles in one CTA, many calls."""
    h, w, labels, _ = make(T, 72, 77000, seed=T)
    first = rfq.linear_ce_alloc(h, w, labels)
    z = h.double() @ w.double().T
    want = torch.logsumexp(z, 1)
    assert ((first[1].double() - want).abs() <= 1e-5 * float((h.double().abs() @ w.double().abs().T).max()) + 1e-5 + 2.0 ** -22 * want.abs()).all()
    for _ in range(20):
        again = rfq.linear_ce_alloc(h, w, labels)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
