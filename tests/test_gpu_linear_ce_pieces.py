"""Gradients of the output head over several pieces of the vocabulary, with the dh product's tiles whole, sliced
along the contraction, or both, and a last piece that is shorter than the others."""
import pytest
import torch

from tests.test_gpu_linear_ce import IGNORE, check, make

pytestmark = pytest.mark.gpu


def reference(h, w, labels, dloss, group=512):
    """As test_gpu_linear_ce.reference (same bounds), rows in groups so that no [T, V] matrix in 64 bits is held."""
    h, w = h.double(), w.double()
    T, V = h.shape[0], w.shape[0]
    top = torch.zeros((), dtype=torch.float64, device=h.device)
    for b in range(0, T, group):
        top = torch.maximum(top, (h[b:b + group].abs() @ w.abs().T).max())
    z_tol = 1e-5 * float(top)
    dh, dh_size = torch.empty_like(h), torch.empty_like(h)
    dw, dw_size = torch.zeros_like(w), torch.zeros_like(w)
    lse_all, loss_all = torch.empty(T, dtype=torch.float64, device=h.device), torch.empty(T, dtype=torch.float64, device=h.device)
    for b in range(0, T, group):
        s = slice(b, min(T, b + group))
        z = h[s] @ w.T
        lse = torch.logsumexp(z, 1)
        counted = labels[s] != IGNORE
        at = torch.where(counted, labels[s], 0)[:, None]
        lse_all[s], loss_all[s] = lse, torch.where(counted, lse - z.gather(1, at)[:, 0], 0.0)
        p = torch.exp(z - lse[:, None])
        g = torch.where(counted, dloss[s].double(), 0.0)[:, None]
        onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
        dz, size = g * (p - onehot), g.abs() * (p + onehot)
        dh[s], dh_size[s] = dz @ w, size @ w.abs()
        dw += dz.T @ h[s]
        dw_size += size.T @ h[s].abs()
    lse_tol = z_tol + 1e-5 + 4 * 2.0 ** -24 * lse_all.abs()
    rel = 2.0 ** -8 + float((lse_tol + z_tol).max()) + 1e-6 + 1e-5
    return {"lse": (lse_all, lse_tol), "loss": (loss_all, lse_tol + z_tol), "dh": (dh, rel * dh_size + 2.0 ** -8 * dh.abs()),
            "dw": (dw, rel * dw_size + 2.0 ** -8 * dw.abs())}


# Four pieces, every tile in nine slices; two pieces, 148 whole tiles and 52 in seven slices; two pieces, 148 whole tiles
# and six in twelve slices, the last of which is empty in the last piece.
@pytest.mark.parametrize("T,D,V", [(4096, 512, 100000), (2500, 5120, 60000), (19523, 368, 8811)])
def test_several_pieces_with_sliced_tiles(rfq, T, D, V):
    h, w, labels, dloss = make(T, D, V, seed=5)
    want = reference(h, w, labels, dloss)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])
    ws = torch.empty(rfq.linear_ce_workspace_bytes(T, D, V, True, True), dtype=torch.uint8, device="cuda")
    ws.fill_(255)   # NaN, wherever what was not written is read
    again = torch.empty_like(dh), torch.empty_like(dw)
    rfq.linear_ce_backward(h, w, labels, lse, dloss, *again, ws)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)
