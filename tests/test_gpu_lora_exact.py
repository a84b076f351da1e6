"""Adapters on whole numbers, where every sum is exact.

x, A, B and dy hold small whole numbers and the scales are powers of two, so s and ds are whole numbers
below 2^15 and every fp32 sum stays below 2^24: each result is the exact value, rounded once to its type.  s and ds need up
to 15 bits, more than one bf16 term has (8) and fewer than two (16).  So a bf16 y or dx whose s or ds went in as
one term is wrong here, and no tolerance hides it behind the rounding of the result.
"""
import pytest
import torch

from tests.test_gpu_lora import BF16, F32, make_ids, run_all

pytestmark = pytest.mark.gpu


def make(M, K, N, r, n, kind, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def whole(top, *shape):
        return torch.randint(-top, top + 1, shape, generator=g, device="cuda").float()

    return {"x": whole(4, M, K).bfloat16(), "a": whole(4, n, r, K).bfloat16(), "b": whole(2, n, N, r).bfloat16(),
            "scale": 2.0 ** torch.randint(-1, 2, (n,), generator=g, device="cuda").float(), "ids": make_ids(kind, M, n, g),
            "base": whole(100, M, N).to(dtype), "dy": whole(1, M, N).bfloat16(), "dx_base": whole(100, M, K).to(dtype)}


def exact(c):
    """{name: value} in float64 (exact: whole numbers and halves far below 2^53)."""
    x, dy = c["x"].double(), c["dy"].double()
    n, r, K = c["a"].shape
    M, N = dy.shape
    y, dx = c["base"].double(), c["dx_base"].double()
    s = torch.zeros((M, r), dtype=torch.float64, device="cuda")
    da, db = torch.zeros((n, r, K), dtype=torch.float64, device="cuda"), torch.zeros((n, N, r), dtype=torch.float64, device="cuda")
    sizes = [0.0]
    for k in range(n):
        rows = torch.nonzero(c["ids"] == k)[:, 0]
        if not rows.numel():
            continue
        a, b, w = c["a"][k].double(), c["b"][k].double(), float(c["scale"][k])
        s[rows] = w * (x[rows] @ a.T)
        ds = w * (dy[rows] @ b)
        y[rows] += s[rows] @ b.T
        dx[rows] += ds @ a
        da[k], db[k] = ds.T @ x[rows], dy[rows].T @ s[rows]
        # the premises: 15 bits for s and ds (in halves), 24 for every sum of products in any order
        assert max(float(s[rows].abs().max()), float(ds.abs().max())) < 2 ** 14
        sizes += [float((s[rows].abs() @ b.abs().T).max()), float((ds.abs() @ a.abs()).max()), float((ds.abs().T @ x[rows].abs()).max()),
                  float((dy[rows].abs().T @ s[rows].abs()).max())]
    assert max(sizes) + 100 < 2 ** 23
    return {"y": y, "hidden": s, "dx": dx, "da": da, "db": db}


SHORT = [(1, 264, 312, 16, 1, "one"), (2, 4096, 520, 16, 2, "mixed"), (40, 1032, 1000, 8, 5, "mixed"), (65, 2056, 264, 128, 2, "runs"), (300, 520, 2056, 24, 40, "mixed")]
LONG = [(68, 8200, 8200, 80, 1, "one"), (300, 4104, 4104, 64, 4, "mixed"), (700, 4104, 4096, 56, 2, "mixed"), (1201, 1032, 5128, 40, 3, "runs"),
        (1111, 5120, 3000, 8, 3, "runs"), (520, 5000, 4008, 128, 12, "mixed"), (2500, 2056, 2568, 24, 4, "runs")]


@pytest.mark.parametrize("M,K,N,r,n,kind", SHORT + LONG)
@pytest.mark.parametrize("out,grad", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
def test_whole_numbers_are_exact(rfq, M, K, N, r, n, kind, out, grad):
    c = make(M, K, N, r, n, kind, M + r, out)
    want = exact(c)
    got = run_all(rfq, c, out, grad)
    for name, t in got.items():
        assert torch.equal(t, want[name].float().to(t.dtype)), name


@pytest.mark.parametrize("M", [65, 97, 129, 161, 255, 257, 383, 1025])
def test_rows_that_end_inside_a_warp(rfq, M):
    """Long batches whose last chunk ends inside a warp: the lanes of the rows past the end have nothing to write and come
    together with the others again at the cluster's barrier."""
    c = make(M, 8200, 8200, 72, 1, "one", M, BF16)
    want = exact(c)
    for _ in range(3):
        got = run_all(rfq, c)
        for name, t in got.items():
            assert torch.equal(t, want[name].float().to(t.dtype)), name
