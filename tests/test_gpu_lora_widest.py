"""Adapters at the widest: 2^20 columns, where s and ds are sums of 2^20 products of one sign, so that an accumulator that
truncates at every step shows.  The bound is that of the other adapter tests (1e-5 of the sum of the products' sizes)."""
import pytest
import torch

from tests.test_gpu_lora import F32, make_ids

pytestmark = pytest.mark.gpu

WIDE = 1 << 20


def check(got, want):
    worst = float(((got - want).abs() / want.clamp(min=1e-30)).max())
    assert worst <= 1e-5, f"off by {worst:.2e} of the sum"


# Few adapters (clusters along the contraction), many (none), and a long batch
@pytest.mark.parametrize("M,r,n,kind", [(3, 16, 2, "mixed"), (40, 8, 40, "mixed"), (300, 8, 64, "mixed"), (300, 24, 90, "mixed"), (300, 16, 1, "one")])
def test_sums_over_2_20_columns(rfq, M, r, n, kind):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + n)
    wide = (0.5 + torch.rand((M, WIDE), generator=g, device="cuda")).bfloat16()
    pool = torch.empty((n, r, WIDE), dtype=torch.bfloat16, device="cuda")
    for part in pool:
        part.copy_((0.5 + torch.rand((r, WIDE), generator=g, device="cuda")) / WIDE)
    ids, scale = make_ids(kind, M, n, g), torch.ones(n, device="cuda")
    small = torch.zeros((n, 8, r), dtype=torch.bfloat16, device="cuda")
    small[:, 0, 0] = 1.0   # dx of one column is ds of one entry
    want = torch.zeros((M, r), dtype=torch.float64, device="cuda")
    for k in range(n):
        rows = torch.nonzero(ids == k)[:, 0]
        if rows.numel():
            want[rows] = wide[rows].double() @ pool[k].double().T
    _, s = rfq.lora_alloc(wide, pool, small, scale, ids, out_dtype=F32, want_hidden=True)
    check(s.double(), want)
    # going back: ds = B^T dy, the same sums
    b = pool.transpose(1, 2).contiguous()
    del pool
    a = torch.zeros((n, r, 8), dtype=torch.bfloat16, device="cuda")
    a[:, 0, 0] = 1.0
    a[:, r - 1, 1] = 1.0
    dx, _, _ = rfq.lora_backward_alloc(None, a, b, scale, ids, wide, None, want_da=False, want_db=False, dx_dtype=F32)
    for col, j in ((0, 0), (1, r - 1)):
        check(dx[:, col].double(), want[:, j])
