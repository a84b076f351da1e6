"""Low-rank adapters beside a projection (rfq_lora, its backward, rfq_linear_lora) against the
definition in float64.

Tolerances, by arithmetic: every product's fp32 sum is off by at most 1e-5 * sum |factors| (the
bound the GEMM's tests use).  s and ds enter the second product rounded: one bf16 term (2^-8) for
bf16 y and dx, two (2^-16) for bf16 dA and dB, three (2^-24) for fp32 results.  Each result is
rounded once: 2^-8 (bf16) or 2^-24 (fp32) of its value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make_ids(kind, M, n, g):
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32, device="cuda")
    if kind == "one":
        return torch.full((M,), n - 1, dtype=torch.int32, device="cuda")
    ids = torch.randint(-1, n + 1, (M,), generator=g, device="cuda", dtype=torch.int32)   # some outside [0, n)
    if kind == "runs":
        ids = torch.sort(ids).values
    return ids


def make(M, K, N, r, n, kind="mixed", seed=0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    return {"x": normal(M, K).bfloat16(), "a": normal(n, r, K, std=K ** -0.5).bfloat16(), "b": normal(n, N, r, std=r ** -0.5).bfloat16(),
            "scale": torch.rand((n,), generator=g, device="cuda") + 0.5, "ids": make_ids(kind, M, n, g),
            "base": normal(M, N).to(dtype), "dy": normal(M, N).bfloat16(), "dx_base": normal(M, K).to(dtype)}


def reference(c, out=BF16, grad=BF16, base=True):
    """{name: (value, tolerance)} adapter by adapter, in float64."""
    x, dy = c["x"].double(), c["dy"].double()
    M, K = x.shape
    n, r, _ = c["a"].shape
    N = c["b"].shape[1]
    dev = x.device
    y = c["base"].double() if base else torch.zeros((M, N), dtype=torch.float64, device=dev)
    dx = c["dx_base"].double() if base else torch.zeros((M, K), dtype=torch.float64, device=dev)
    ty, tx = torch.zeros_like(y), torch.zeros_like(dx)
    s, ts = (torch.zeros((M, r), dtype=torch.float64, device=dev) for _ in range(2))
    da, ta = (torch.zeros((n, r, K), dtype=torch.float64, device=dev) for _ in range(2))
    db, tb = (torch.zeros((n, N, r), dtype=torch.float64, device=dev) for _ in range(2))
    q_out, q_grad = (2.0 ** -8 if out == BF16 else 2.0 ** -24), (2.0 ** -16 if grad == BF16 else 2.0 ** -24)
    for k in range(n):
        rows = torch.nonzero(c["ids"] == k)[:, 0]
        a, b, w = c["a"][k].double(), c["b"][k].double(), float(c["scale"][k])
        xa, da_ = x[rows], dy[rows]
        sk, sk_t = w * (xa @ a.T), 1e-5 * w * (xa.abs() @ a.abs().T) + 1e-30
        dk, dk_t = w * (da_ @ b), 1e-5 * w * (da_.abs() @ b.abs()) + 1e-30
        s[rows], ts[rows] = sk, sk_t + 2.0 ** -23 * sk.abs()
        y[rows] += sk @ b.T
        ty[rows] = (sk_t + (q_out + 1e-5) * sk.abs()) @ b.abs().T
        dx[rows] += dk @ a
        tx[rows] = (dk_t + (q_out + 1e-5) * dk.abs()) @ a.abs()
        da[k], ta[k] = dk.T @ xa, (dk_t + (q_grad + 1e-5) * dk.abs()).T @ xa.abs()
        db[k], tb[k] = da_.T @ sk, da_.abs().T @ (sk_t + (q_grad + 1e-5) * sk.abs())
    u_out, u_grad = (2.0 ** -8 if out == BF16 else 2.0 ** -24), (2.0 ** -8 if grad == BF16 else 2.0 ** -24)
    # the fp32 sum with the base is rounded too before a bf16 result is
    return {"y": (y, ty * 1.01 + (u_out + 2.0 ** -23) * y.abs()), "dx": (dx, tx * 1.01 + (u_out + 2.0 ** -23) * dx.abs()), "hidden": (s, ts),
            "da": (da, ta * 1.01 + u_grad * da.abs()), "db": (db, tb * 1.01 + u_grad * db.abs())}


def check(name, got, want):
    ref, tol = want
    assert got.shape == ref.shape
    assert torch.isfinite(got.float()).all(), f"{name}: not finite"
    err = (got.double() - ref).abs()
    over = (err - tol).max() if err.numel() else torch.zeros(())
    assert float(over) <= 0, f"{name}: off by {float(err.max()):.3e}, {float(over):.3e} over the bound"


def run_all(rfq, c, out=BF16, grad=BF16, base=True):
    y, hidden = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=c["base"] if base else None, out_dtype=out, want_hidden=True)
    dx, da, db = rfq.lora_backward_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], hidden, dx_base=c["dx_base"] if base else None,
                                         dx_dtype=out, grad_dtype=grad)
    return {"y": y, "hidden": hidden, "dx": dx, "da": da, "db": db}


SHAPES = [(1, 8, 8, 8, 1, "one"), (1, 64, 40, 16, 3, "mixed"), (2, 136, 264, 24, 5, "mixed"), (15, 264, 8, 32, 2, "runs"),
          (16, 512, 520, 16, 16, "mixed"), (17, 72, 1032, 40, 4, "mixed"), (64, 1032, 256, 64, 1, "one"), (65, 256, 136, 128, 2, "runs"),
          (128, 200, 200, 8, 40, "mixed"), (129, 520, 72, 72, 3, "runs"), (300, 264, 312, 16, 200, "mixed"), (300, 264, 312, 128, 2, "mixed"),
          (700, 384, 1000, 56, 3, "runs"), (1000, 128, 136, 8, 6, "mixed"), (2500, 64, 72, 16, 4, "runs"), (5000, 40, 136, 32, 300, "mixed"),
          (200, 8, 8, 8, 1, "one"), (200, 16, 24, 128, 1, "one"), (140, 72, 8, 40, 2, "mixed"), (257, 2056, 64, 24, 40, "runs"),
          (1500, 1032, 264, 104, 40, "mixed"), (33, 200, 136, 120, 4, "mixed")]


@pytest.mark.parametrize("M,K,N,r,n,kind", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward_and_gradients(rfq, M, K, N, r, n, kind, dtype):
    c = make(M, K, N, r, n, kind, seed=M + r, dtype=dtype)
    want = reference(c, dtype, dtype)
    got = run_all(rfq, c, dtype, dtype)
    for name, t in got.items():
        assert name == "hidden" or t.dtype == dtype
        check(name, t, want[name])


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_a_base(rfq, M, dtype):
    c = make(M, 264, 312, 16, 4, seed=5)
    want = reference(c, dtype, dtype, base=False)
    for name, t in run_all(rfq, c, dtype, dtype, base=False).items():
        check(name, t, want[name])


@pytest.mark.parametrize("M", [5, 333])
def test_in_place_is_the_same_and_leaves_rows_without_an_adapter(rfq, M):
    c = make(M, 264, 312, 16, 4, seed=6)
    c["ids"][0] = -1
    out = run_all(rfq, c)
    y, dx = c["base"].clone(), c["dx_base"].clone()
    y[0] = float("nan")   # an untouched row keeps its bits, whatever they are
    bits = y[0].view(torch.int16).clone()
    ws = torch.empty(rfq.lora_workspace_bytes(M, 264, 312, 16, 4, backward=True), dtype=torch.uint8, device="cuda")
    rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], y, ws, base=y)
    rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], out["hidden"], ws, dx=dx, dx_base=dx)
    assert torch.equal(y[0].view(torch.int16), bits)
    assert torch.equal(y[1:], out["y"][1:]) and torch.equal(dx, out["dx"])


@pytest.mark.parametrize("kind", ["none", "one"])
def test_no_adapter_or_one_for_all(rfq, kind):
    c = make(200, 128, 136, 8, 3, kind, seed=7)
    want = reference(c)
    got = run_all(rfq, c)
    for name, t in got.items():
        check(name, t, want[name])
    if kind == "none":
        assert torch.equal(got["y"], c["base"]) and torch.equal(got["dx"], c["dx_base"])
        assert not got["hidden"].any() and not got["da"].any() and not got["db"].any()
    else:
        assert not got["da"][:2].any() and not got["db"][:2].any() and got["da"][2].any()


def test_row_order_does_not_change_a_row(rfq):
    c = make(100, 264, 312, 16, 4, seed=8)
    perm = torch.randperm(100, device="cuda")
    y = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=c["base"])
    z = rfq.lora_alloc(c["x"][perm], c["a"], c["b"], c["scale"], c["ids"][perm], base=c["base"][perm])
    assert torch.equal(y[perm], z)


@pytest.mark.parametrize("wants", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
def test_each_gradient_alone_is_the_same_bits(rfq, wants):
    c = make(300, 264, 312, 16, 4, seed=9)
    all_ = run_all(rfq, c)
    some = rfq.lora_backward_alloc(c["x"] if wants[1] else None, c["a"], c["b"], c["scale"], c["ids"], c["dy"], all_["hidden"] if wants[2] else None,
                                   dx_base=c["dx_base"], want_dx=wants[0], want_da=wants[1], want_db=wants[2])
    for w, t, name in zip(wants, some, ("dx", "da", "db")):
        assert (t is not None) == w and (t is None or torch.equal(t, all_[name]))


def test_values_that_are_not_finite_stay_where_they_are(rfq):
    c = make(150, 128, 136, 24, 3, "mixed", seed=10)
    c["ids"][c["ids"] == 1] = 0
    clean = run_all(rfq, c)
    rows0 = c["ids"] == 0
    bad = int(torch.nonzero(c["ids"] == 2)[0])
    c["a"][1] = float("nan")        # an adapter that no row uses
    c["b"][1] = float("inf")
    c["x"][bad, 3] = float("inf")   # a row of adapter 2
    c["dy"][bad, 5] = float("nan")
    got = run_all(rfq, c)
    keep = torch.ones(150, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for name in ("y", "dx", "hidden"):
        assert torch.equal(got[name][keep], clean[name][keep])
    assert not torch.isfinite(got["y"][bad].float()).any() and not torch.isfinite(got["dx"][bad].float()).any()
    assert torch.equal(got["da"][0], clean["da"][0]) and torch.equal(got["db"][0], clean["db"][0]) and rows0.any()
    assert not got["da"][1].any() and not got["db"][1].any()


def test_gradients_are_the_differences(rfq):
    """dx, dA, dB along random directions against central differences of sum(y * dy) in float64 (the map is
    bilinear: the differences are exact but for rounding)."""
    c = make(60, 128, 136, 16, 3, seed=12, dtype=F32)
    got = run_all(rfq, c, F32, F32, base=False)
    want = reference(c, F32, F32, base=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def total(x, a, b):
        f = 0.0
        for k in range(3):
            rows = c["ids"] == k
            f = f + float(c["scale"][k]) * ((x[rows] @ a[k].T) @ b[k].T * c["dy"][rows].double()).sum()
        return float(f)

    at = {"dx": c["x"].double(), "da": c["a"].double(), "db": c["b"].double()}
    for name in at:
        u = torch.randn(at[name].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = ({**at, name: at[name] + e * u} for e in (1e-3, -1e-3))
        diff = (total(plus["dx"], plus["da"], plus["db"]) - total(minus["dx"], minus["da"], minus["db"])) / 2e-3
        tol = float((want[name][1] * u.abs()).sum()) + 1e-8 * abs(diff) + 1e-8
        assert abs(float((got[name].double() * u).sum()) - diff) <= tol


def test_repeats_bit_for_bit_and_leaves_its_inputs(rfq):
    c = make(700, 520, 264, 32, 9, seed=13)
    kept = {k: t.clone() for k, t in c.items()}
    first = run_all(rfq, c)
    for _ in range(5):
        again = run_all(rfq, c)
        assert all(torch.equal(first[k], again[k]) for k in first)
    assert all(torch.equal(kept[k], c[k]) for k in c)


def test_nothing_outside_the_outputs_is_written(rfq):
    M, K, N, r, n = 77, 72, 136, 24, 3
    c = make(M, K, N, r, n, seed=14)
    pad = 64

    def fenced(shape, dtype):
        size = 1
        for d in shape:
            size *= d
        t = torch.full((size + 2 * pad,), 7.0, dtype=dtype, device="cuda")
        return t, t[pad:pad + size].view(shape)

    outs = {"y": fenced((M, N), BF16), "hidden": fenced((M, r), F32), "dx": fenced((M, K), BF16), "da": fenced((n, r, K), BF16),
            "db": fenced((n, N, r), BF16)}
    need = rfq.lora_workspace_bytes(M, K, N, r, n, backward=True)
    ws_f = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")
    ws = ws_f[256:256 + need]
    rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], outs["y"][1], ws, base=c["base"], hidden=outs["hidden"][1])
    rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], outs["hidden"][1], ws, dx=outs["dx"][1], dx_base=c["dx_base"],
                      da=outs["da"][1], db=outs["db"][1])
    torch.cuda.synchronize()
    want = reference(c)
    for name, (f, t) in outs.items():
        assert (f[:pad] == 7).all() and (f[-pad:] == 7).all(), name
        check(name, t, want[name])
    assert (ws_f[:256] == 165).all() and (ws_f[256 + need:] == 165).all()


def test_captured_graph_follows_its_inputs(rfq):
    M, K, N, r, n = 40, 264, 312, 16, 6
    c = make(M, K, N, r, n, seed=15)
    y, hidden = torch.empty_like(c["base"]), torch.empty((M, r), device="cuda")
    dx, da, db = torch.empty_like(c["dx_base"]), torch.empty_like(c["a"]), torch.empty_like(c["b"])
    ws = torch.empty(rfq.lora_workspace_bytes(M, K, N, r, n, backward=True), dtype=torch.uint8, device="cuda")

    def step():
        rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], y, ws, base=c["base"], hidden=hidden)
        rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], hidden, ws, dx=dx, dx_base=c["dx_base"], da=da, db=db)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, kind in ((16, "mixed"), (17, "runs"), (18, "none")):
        for name, t in make(M, K, N, r, n, kind, seed=seed).items():
            c[name].copy_(t)
        graph.replay()
        want = reference(c)
        for name, t in (("y", y), ("hidden", hidden), ("dx", dx), ("da", da), ("db", db)):
            check(name, t, want[name])


def test_another_stream(rfq):
    c = make(90, 264, 312, 16, 6, seed=19)
    base = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=c["base"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=c["base"], stream=side)
    side.synchronize()
    assert torch.equal(base, got)


def test_offsets_past_32_bits(rfq):
    """More than 2^31 elements of base and output: the last rows are those of a small call on them."""
    M, K, N, r, n = 66000, 64, 32776, 8, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    c = make(300, K, N, r, n, "runs", seed=23)
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    base = torch.zeros((M, N), dtype=BF16, device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    x[-300:], base[-300:], ids[-300:] = c["x"], c["base"], c["ids"]
    y = rfq.lora_alloc(x, c["a"], c["b"], c["scale"], ids, base=base)
    want = reference(c)
    check("y", y[-300:], want["y"])
    assert not y[:-300].any()
    # the same through the gradients: dy is the wide one
    hidden = torch.zeros((M, r), device="cuda")
    hidden[-300:] = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], want_hidden=True)[1]
    base.zero_()
    base[-300:] = c["dy"]
    dx, da, db = rfq.lora_backward_alloc(x, c["a"], c["b"], c["scale"], ids, base, hidden)
    want = reference(c, base=False)
    check("dx", dx[-300:], want["dx"])
    check("da", da, want["da"])
    check("db", db, want["db"])


def test_no_rows(rfq):
    c = make(0, 64, 72, 8, 2)
    out = run_all(rfq, c)
    assert out["y"].shape == (0, 72) and not out["da"].any() and not out["db"].any()


@pytest.mark.parametrize("M", [1, 16, 40, 200, 600])
@pytest.mark.parametrize("out", [BF16, F32])
def test_linear_with_adapters_is_linear_plus_adapters(rfq, M, out):
    K, N, r, n = 512, 520, 16, 5
    c = make(M, K, N, r, n, seed=20)
    qw = rfq.quantize_weight_alloc((torch.randn((N, K), device="cuda") * 0.05).bfloat16())
    y = rfq.linear_alloc(c["x"], qw, out_dtype=out)
    want = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=y)
    got, hidden = rfq.linear_lora_alloc(c["x"], qw, c["a"], c["b"], c["scale"], c["ids"], out_dtype=out, want_hidden=True)
    assert torch.equal(got, want)
    check("hidden", hidden, reference(c)["hidden"])
    # rows without an adapter are the projection's own
    assert torch.equal(got[(c["ids"] < 0) | (c["ids"] >= n)], y[(c["ids"] < 0) | (c["ids"] >= n)])


def test_binding_refuses_what_the_kernel_cannot_read(rfq):
    c = make(16, 64, 72, 8, 2)
    y = torch.empty_like(c["base"])
    ws = torch.empty(rfq.lora_workspace_bytes(16, 64, 72, 8, 2, backward=True), dtype=torch.uint8, device="cuda")
    good = dict(x=c["x"], a=c["a"], b=c["b"], scale=c["scale"], ids=c["ids"], y=y, workspace=ws)
    rfq.lora(**good)
    for name, bad in (("x", c["x"].float()), ("x", c["x"][:, :32]), ("a", c["a"][:, :, :32].contiguous()), ("a", c["a"].cpu()),
                      ("b", c["b"].transpose(1, 2)), ("scale", c["scale"].double()), ("ids", c["ids"].long()), ("ids", c["ids"][:3]),
                      ("y", y.half()), ("y", y[:, ::2]), ("workspace", ws.float()), ("base", c["base"].float()), ("hidden", torch.empty(16, 8))):
        with pytest.raises(rfq.RFQError) as e:
            rfq.lora(**{**good, name: bad})
        assert e.value.status == 1, name
    with pytest.raises(rfq.RFQError) as e:
        rfq.lora(**{**good, "workspace": ws[:16]})
    assert e.value.status == 7
