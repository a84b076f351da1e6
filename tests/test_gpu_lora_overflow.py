"""Rank vectors at the end of the range: s and ds of the adapters enter the second product as sums of bf16 terms,
and what does not fit a term must not turn the others into NaN."""
import pytest
import torch

from tests.test_gpu_lora import BF16, F32

pytestmark = pytest.mark.gpu


# short forward and backward, long forward and backward, ds of a long batch by groups
@pytest.mark.parametrize("M,K,N,r", [(3, 64, 40, 16), (3, 64, 40, 24), (300, 4104, 4104, 64), (300, 4104, 4104, 8), (1201, 1032, 5128, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("large", [False, True])
def test_infinite_and_largest_rank_vectors(rfq, M, K, N, r, dtype, large):
    """One entry of s (and of ds) is infinite, or within 2^-9 of the largest fp32 number (so that bf16 rounds it to infinity): y (dx) is
    infinite with the signs of B (A), or their finite product."""
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    a = torch.zeros((1, r, K), dtype=BF16, device="cuda")
    b = torch.zeros((1, N, r), dtype=BF16, device="cuda")
    dy = torch.zeros((M, N), dtype=BF16, device="cuda")
    row, j = M - 1, r - 3
    sign = torch.where(torch.arange(max(K, N), device="cuda") % 3 == 0, -1.0, 1.0)
    b[0, :, j] = sign[:N] * 2.0 ** -20
    a[0, j, :] = sign[:K] * 2.0 ** -20
    if large:   # past the last bf16 number (the first product) by more than half a step, and below fp32's end
        a[0, j, 0], a[0, j, 1], x[row, 0], x[row, 1] = 1.9921875, 1.0078125, 2.0 ** 127, 2.0 ** 119
        b[0, 0, j], b[0, 1, j], dy[row, 0], dy[row, 1] = 1.9921875, 1.0078125, 2.0 ** 127, 2.0 ** 119
        size = 2.0 ** 127 * 1.9921875 + 2.0 ** 119 * 1.0078125
        assert torch.isinf(torch.tensor(size).bfloat16()) and torch.isfinite(torch.tensor(size))
    else:
        a[0, j, 0], x[row, 0], b[0, 0, j], dy[row, 0] = 4.0, 2.0 ** 127, 4.0, 2.0 ** 127
        size = float("inf")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    scale = torch.ones(1, device="cuda")
    y, hidden = rfq.lora_alloc(x, a, b, scale, ids, out_dtype=dtype, want_hidden=True)
    dx, _, _ = rfq.lora_backward_alloc(x, a, b, scale, ids, dy, hidden, want_da=False, want_db=False, dx_dtype=dtype)
    assert float(hidden[row, j]) == size and not hidden[:row].any()
    for got, w in ((y, b[0, :, j]), (dx, a[0, j])):
        assert not got[:row].any()
        small = w.abs() < 2.0 ** -10   # the others times such an s leave the range themselves
        want = size * w[small].double()
        assert torch.equal(torch.sign(got[row][small].float()), torch.sign(want).float())
        if large:
            assert ((got[row][small].double() - want).abs() <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -22) * want.abs()).all()
        else:
            assert torch.isinf(got[row][small]).all()


@pytest.mark.parametrize("M,K,N,r", [(3, 64, 40, 16), (1201, 1032, 5128, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_infinite_rank_vectors(rfq, M, K, N, r, dtype):
    """dB = dy s^T where one entry of s is infinite, dA = ds x^T where one of ds is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    x = torch.ones((M, K), dtype=BF16, device="cuda")
    dy = torch.ones((M, N), dtype=BF16, device="cuda")
    a = torch.randn((1, r, K), generator=g, device="cuda").bfloat16()
    b = torch.randn((1, N, r), generator=g, device="cuda").bfloat16()
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    scale = torch.ones(1, device="cuda")
    hidden = torch.randn((M, r), generator=g, device="cuda")
    hidden[1, 5], hidden[2, 5] = float("-inf"), 0.0
    b[0, 0, 4], b[0, 1, 4], dy[2, 0] = 4.0, 1.0, 2.0 ** 127   # ds[2][4] leaves the range, the other entries of row 2 ...
    b[0, 0, :4] = 0.0
    b[0, 0, 5:] = 0.0                                         # ... do not see it
    _, da, db = rfq.lora_backward_alloc(x, a, b, scale, ids, dy, hidden, want_dx=False, grad_dtype=dtype)
    assert (da[0, 4] == float("inf")).all()
    rest = [i for i in range(r) if i != 4]
    assert torch.isfinite(da[0, rest].float()).all()
    assert (db[0, :, 5] == float("-inf")).all()
    assert torch.isfinite(db[0][:, [i for i in range(r) if i != 5]].float()[1:]).all()
