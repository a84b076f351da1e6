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


@pytest.mark.parametrize("T", [8, 20, 200])
@pytest.mark.parametrize("D", [4096, 65536])
def test_certain_labels(rfq, T, D):
    """Rows whose label has p = 1 - 1e-3: the label's term of the gradient is held to its own size, 1 - p.

    By arithmetic: 1 - p is off by 2 |dz| (1 - p) where every logit is off by dz <= 1e-5 sum |h w| in the same way in both
    passes, and by p (2 |lse| 2^-24 + 2^-22): lse is kept in fp32, scaled by log2 e in fp32, and the exponential has 2^-22.
    (The two passes' logits differing by 3e-6 of their size, as sums of 4096 and of 1024 terms do, would be 4e-5 here: 4 % of 1 - p.)
    dz is rounded to bf16 (2^-8), dw and dh are fp32 sums (1e-5 of their terms) rounded once."""
    V, y0 = 300, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    h = (0.5 + torch.rand((T, D), generator=g, device="cuda")).bfloat16()
    w = torch.randn((V, D), generator=g, device="cuda") / D ** 0.5
    w[y0] = 12.8 / D * (0.5 + torch.rand((D,), generator=g, device="cuda"))
    w = w.bfloat16()
    labels = torch.full((T,), y0, device="cuda")
    dloss = torch.ones(T, device="cuda")
    h64, w64 = h.double(), w.double()
    z = h64 @ w64.T
    lse64 = torch.logsumexp(z, 1)
    p = torch.exp(z - lse64[:, None])
    dz = p.clone()
    others = p.clone()
    others[:, y0] = 0
    dz[:, y0] = -others.sum(1)   # p - 1 without the cancellation
    assert ((-dz[:, y0] > 1e-4) & (-dz[:, y0] < 1e-2)).all()
    z_tol = 1e-5 * float((h64.abs() @ w64.abs().T).max())
    term = (2.0 ** -8 + 2 * z_tol + 2e-5) * dz.abs() + p * (2 * lse64.abs()[:, None] * 2.0 ** -24 + 2.0 ** -22)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    check("dw", dw, (dz.T @ h64, term.T @ h64.abs() + 2.0 ** -8 * (dz.T @ h64).abs()))
    check("dh", dh, (dz @ w64, term @ w64.abs() + 2.0 ** -8 * (dz @ w64).abs()))


def test_head_gradient_of_very_many_rows(rfq):
    """2^24 - 3 rows, as many as a call takes: with equal logits dz is 1/64 (exact in bf16) for all entries but the label's, and
    all terms of dw have one sign.  p is off by 1e-5 at most (lse of 64 equal logits), dw is rounded once, and its
    sum over the rows may lose 2^-12 (one accumulator that truncates at every step loses 1 %)."""
    T, D, V = (1 << 24) - 3, 8, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    h = (0.5 + torch.rand((T, D), generator=g, device="cuda")).bfloat16()
    w = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    labels = torch.zeros(T, dtype=torch.int64, device="cuda")
    lse = torch.full((T,), 64.0, device="cuda").log_()
    dloss = torch.ones(T, device="cuda")
    _, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss, want_dh=False)
    total = sum(part.double().sum(0) for part in h.split(1 << 22))
    want = total[None, :] * torch.cat([torch.full((1, 1), 1 / 64 - 1.0), torch.full((V - 1, 1), 1 / 64)]).double().cuda()
    assert ((dw.double() - want).abs() <= (2.0 ** -8 + 1e-5 + 2.0 ** -12) * want.abs()).all()


@pytest.mark.parametrize("T", [32868, 65537])
def test_certain_labels_of_the_last_rows(rfq, T):
    """The forward pass takes long batches in groups of rows, and a last group of few rows is still summed as the backward pass sums
    it.  Logits near 100, of which the label's leads by 12.6: a difference of 1e-6 of the logits between the passes would be 10 % of
    1 - p.  Only the last 100 rows count (or the one past two full groups).  Same bounds as in test_certain_labels."""
    D, V, y0 = 4096, 300, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    h = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    for part in h.split(8192):
        part.copy_(0.5 + torch.rand(part.shape, generator=g, device="cuda"))
    w = torch.randn((V, D), generator=g, device="cuda") / D ** 0.5 + 87.2 / D
    w[y0] = 100.0 / D * (0.5 + torch.rand((D,), generator=g, device="cuda"))
    w = w.bfloat16()
    last = slice(T - (T % 32768 if T % 32768 > 1 else 1), T)
    labels = torch.full((T,), IGNORE, device="cuda")
    labels[last] = y0
    h64, w64 = h[last].double(), w.double()
    z = h64 @ w64.T
    lse64 = torch.logsumexp(z, 1)
    p = torch.exp(z - lse64[:, None])
    dz, others = p.clone(), p.clone()
    others[:, y0] = 0
    dz[:, y0] = -others.sum(1)
    assert ((-dz[:, y0] > 1e-5) & (-dz[:, y0] < 1e-1)).all()
    # every logit is off by dz in the same way in both passes, those of a row by nearly the same share: 2 dz of the logits' spread
    spread = 1e-5 * float((z.amax(1) - z.amin(1)).max())
    term = (2.0 ** -8 + 2 * spread + 2e-5) * dz.abs() + p * (2 * lse64.abs()[:, None] * 2.0 ** -24 + 2.0 ** -22)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    _, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, torch.ones(T, device="cuda"), want_dh=False)
    check("dw", dw, (dz.T @ h64, term.T @ h64.abs() + 2.0 ** -8 * (dz.T @ h64).abs()))
