"""2^24 rows, the most that a call takes, of narrow matrices: adapters and the output head's loss, with their gradients."""
import pytest
import torch

from tests.test_gpu_lora import BF16, check, make, reference, run_all

pytestmark = pytest.mark.gpu

ROWS = 1 << 24


@pytest.mark.parametrize("n,kind", [(1, "one"), (3, "runs")])
def test_adapters(rfq, n, kind):
    c = make(ROWS, 8, 8, 8, n, kind, seed=n)
    want = reference(c)
    for name, t in run_all(rfq, c).items():
        check(name, t, want[name])


def test_output_head(rfq):
    """Row by row against float64 (bounds as in test_gpu_linear_ce); dw's sums are 2^24 terms of both signs: one bf16 rounding, dz's
    roundings and 2^-12 of the terms, see test_head_gradient_of_very_many_rows."""
    D, V = 8, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn((ROWS, D), generator=g, device="cuda").bfloat16()
    w = (torch.randn((V, D), generator=g, device="cuda") * 0.5).bfloat16()
    labels = torch.randint(-100, V, (ROWS,), generator=g, device="cuda")
    labels = torch.where(labels < 0, -100, labels)
    dloss = torch.rand((ROWS,), generator=g, device="cuda") + 0.1
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    want_dw = torch.zeros((V, D), dtype=torch.float64, device="cuda")
    size_dw = torch.zeros_like(want_dw)
    w64 = w.double()
    for b in range(0, ROWS, 1 << 22):
        s = slice(b, b + (1 << 22))
        h64 = h[s].double()
        z = h64 @ w64.T
        lse64 = torch.logsumexp(z, 1)
        counted = labels[s] >= 0
        at = torch.where(counted, labels[s], 0)[:, None]
        tol = 1e-5 * float((h64.abs() @ w64.abs().T).max()) + 1e-5 + 4 * 2.0 ** -24 * lse64.abs()
        assert ((lse[s].double() - lse64).abs() <= tol).all()
        assert ((loss[s].double() - torch.where(counted, lse64 - z.gather(1, at)[:, 0], 0.0)).abs() <= 2 * tol).all()
        p = torch.exp(z - lse64[:, None])
        onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
        gd = torch.where(counted, dloss[s].double(), 0.0)[:, None]
        dz, size = gd * (p - onehot), gd * (p + onehot)
        rel = 2.0 ** -8 + 2 * float(tol.max()) + 1e-5
        assert ((dh[s].double() - dz @ w64).abs() <= rel * (size @ w64.abs()) + 2.0 ** -8 * (dz @ w64).abs()).all()
        want_dw += dz.T @ h64
        size_dw += size.T @ h64.abs()
    assert ((dw.double() - want_dw).abs() <= (rel + 2.0 ** -12) * size_dw + 2.0 ** -8 * want_dw.abs()).all()
