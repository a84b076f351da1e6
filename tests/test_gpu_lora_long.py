"""Adapters over long batches: sizes from which the two products go by chunks of 128 neighbouring rows, forward (about
rows x (rank + 8) x (K + N) above 3.3e8), backward (rows x rank x (K + N) above 6e7), and there with ds by groups (up to
20000 rows x rank) or by chunks too, and the adapters' gradients by stages of 64 rows of one adapter (from rank 24 and
96 rows for each adapter on, or one adapter and 6000 rows).  Same definition, same bounds as for short ones."""
import pytest
import torch

from tests.test_gpu_lora import BF16, F32, check, make, reference, run_all

pytestmark = pytest.mark.gpu

LONG = [(2500, 2056, 2568, 24, 4, "runs"), (1201, 1032, 5128, 40, 3, "runs"), (700, 4104, 4096, 56, 2, "mixed"), (2000, 2048, 2056, 128, 1, "one"),
        (520, 5000, 4008, 128, 12, "mixed"), (300, 4104, 4104, 64, 4, "mixed"), (1111, 5120, 3000, 8, 3, "runs"), (129, 8008, 8200, 72, 2, "runs"),
        (4100, 3080, 1544, 16, 9, "runs"), (68, 8200, 8200, 80, 1, "one"),
        (8200, 520, 264, 16, 1, "one"), (5000, 8200, 8200, 24, 2, "mixed"), (3000, 264, 2056, 104, 3, "runs")]


@pytest.fixture(scope="module")
def rfq():
    import block_scaled_gemm_rfq_b200 as m
    yield m
    torch.cuda.synchronize()
    m.check_device_error()


@pytest.mark.parametrize("M,K,N,r,n,kind", LONG)
@pytest.mark.parametrize("out,grad", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
def test_forward_and_gradients(rfq, M, K, N, r, n, kind, out, grad):
    c = make(M, K, N, r, n, kind, seed=M + r, dtype=out)
    want = reference(c, out, grad)
    for name, t in run_all(rfq, c, out, grad).items():
        check(name, t, want[name])


SOME = [LONG[1], LONG[2], LONG[5], LONG[6], LONG[12]]


@pytest.mark.parametrize("M,K,N,r,n,kind", SOME)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_a_base(rfq, M, K, N, r, n, kind, dtype):
    c = make(M, K, N, r, n, kind, seed=5)
    c["ids"][3::7] = -1
    want = reference(c, dtype, dtype, base=False)
    for name, t in run_all(rfq, c, dtype, dtype, base=False).items():
        check(name, t, want[name])


@pytest.mark.parametrize("M,K,N,r,n,kind", SOME)
def test_in_place_is_the_same_and_leaves_rows_without_an_adapter(rfq, M, K, N, r, n, kind):
    c = make(M, K, N, r, n, kind, seed=6)
    c["ids"][:130] = n
    c["ids"][140] = -5
    out = run_all(rfq, c)
    ws = torch.empty(rfq.lora_workspace_bytes(M, K, N, r, n, backward=True), dtype=torch.uint8, device="cuda")
    y, dx = c["base"].clone(), c["dx_base"].clone()
    y[7] = float("nan")
    bits = y[7].view(torch.int16).clone()
    ws.fill_(255)   # NaN, wherever what is not written is read
    rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], y, ws, base=y)
    ws.fill_(255)
    rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], out["hidden"], ws, dx=dx, dx_base=dx)
    assert torch.equal(y[7].view(torch.int16), bits)
    y[7] = out["y"][7]
    assert torch.equal(y, out["y"]) and torch.equal(dx, out["dx"])
    assert torch.equal(y[140], c["base"][140]) and torch.equal(dx[:130], c["dx_base"][:130])


@pytest.mark.parametrize("M,K,N,r,n,kind", SOME)
def test_each_gradient_alone_is_the_same_bits(rfq, M, K, N, r, n, kind):
    c = make(M, K, N, r, n, kind, seed=9)
    all_ = run_all(rfq, c)
    for wants in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        some = rfq.lora_backward_alloc(c["x"] if wants[1] else None, c["a"], c["b"], c["scale"], c["ids"], c["dy"], all_["hidden"] if wants[2] else None,
                                       dx_base=c["dx_base"], want_dx=wants[0], want_da=wants[1], want_db=wants[2])
        for w, t, name in zip(wants, some, ("dx", "da", "db")):
            assert (t is not None) == w and (t is None or torch.equal(t, all_[name])), name


@pytest.mark.parametrize("M,K,N,r,n,kind", [LONG[0], LONG[5], LONG[6], LONG[12]])
def test_values_that_are_not_finite_stay_where_they_are(rfq, M, K, N, r, n, kind):
    c = make(M, K, N, r, n, kind, seed=10)
    c["ids"][c["ids"] == 1] = 0
    clean = run_all(rfq, c)
    bad = int(torch.nonzero(c["ids"] == 2)[0])
    c["a"][1] = float("nan")        # an adapter that no row uses
    c["b"][1] = float("inf")
    c["x"][bad, 3] = float("inf")   # a row of adapter 2
    c["dy"][bad, 5] = float("nan")
    without = c["ids"] < 0          # rows without an adapter
    c["x"][without] = float("nan")
    c["dy"][without] = float("inf")
    got = run_all(rfq, c)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for name in ("y", "dx", "hidden"):
        assert torch.equal(got[name][keep], clean[name][keep]), name
    assert not torch.isfinite(got["y"][bad].float()).any() and not torch.isfinite(got["dx"][bad].float()).any()
    assert torch.equal(got["da"][0], clean["da"][0]) and torch.equal(got["db"][0], clean["db"][0])
    assert not got["da"][1].any() and not got["db"][1].any()


@pytest.mark.parametrize("M,K,N,r,n,kind", SOME)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nothing_outside_the_outputs_is_written(rfq, M, K, N, r, n, kind, dtype):
    c = make(M, K, N, r, n, kind, seed=14, dtype=dtype)
    pad = 64

    def fenced(shape, t):
        size = 1
        for d in shape:
            size *= d
        f = torch.full((size + 2 * pad,), 7.0, dtype=t, device="cuda")
        return f, f[pad:pad + size].view(shape)

    outs = {"y": fenced((M, N), dtype), "hidden": fenced((M, r), F32), "dx": fenced((M, K), dtype), "da": fenced((n, r, K), dtype),
            "db": fenced((n, N, r), dtype)}
    for backward in (False, True):
        need = rfq.lora_workspace_bytes(M, K, N, r, n, backward=backward)
        fence = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")
        ws = fence[256:256 + need]
        if not backward:
            rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], outs["y"][1], ws, base=c["base"], hidden=outs["hidden"][1])
        else:
            rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], outs["hidden"][1], ws, dx=outs["dx"][1],
                              dx_base=c["dx_base"], da=outs["da"][1], db=outs["db"][1])
        torch.cuda.synchronize()
        assert (fence[:256] == 165).all() and (fence[256 + need:] == 165).all()
    want = reference(c, dtype, dtype)
    for name, (f, t) in outs.items():
        assert (f[:pad] == 7).all() and (f[-pad:] == 7).all(), name
        check(name, t, want[name])


def test_repeats_bit_for_bit(rfq):
    for case in SOME:
        c = make(*case, seed=13)
        first = run_all(rfq, c)
        for _ in range(3):
            again = run_all(rfq, c)
            assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("M,K,N,r,n,kind", [LONG[1], LONG[5], LONG[6]])
def test_two_captured_graphs_follow_their_inputs_at_once(rfq, M, K, N, r, n, kind):
    """Two graphs of a forward and a backward pass, each with tensors and a workspace of its own, replayed on two streams
    at the same time with other inputs than they were captured with."""
    names = ("y", "hidden", "dx", "da", "db")
    sets = []
    for i in range(2):
        c = make(M, K, N, r, n, kind, seed=50 + i)
        o = {"y": torch.empty_like(c["base"]), "hidden": torch.empty((M, r), device="cuda"), "dx": torch.empty_like(c["dx_base"]),
             "da": torch.empty_like(c["a"]), "db": torch.empty_like(c["b"])}
        ws = torch.empty(rfq.lora_workspace_bytes(M, K, N, r, n, backward=True), dtype=torch.uint8, device="cuda")

        def run(c=c, o=o, ws=ws):
            rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], o["y"], ws, base=c["base"], hidden=o["hidden"])
            rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], o["hidden"], ws, dx=o["dx"], dx_base=c["dx_base"], da=o["da"],
                              db=o["db"])

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        sets.append((c, o, graph, torch.cuda.Stream(), ws))   # a graph's workspace lives as long as the graph
    want = []
    for i, (c, o, _, _, _) in enumerate(sets):
        new = make(M, K, N, r, n, "mixed" if kind == "runs" else "runs", seed=60 + i)
        for k in c:
            c[k].copy_(new[k])
        want.append(run_all(rfq, new))
        for t in o.values():
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for _, _, graph, stream, _ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, o, _, _, _), w in zip(sets, want):
        assert [k for k in names if not torch.equal(o[k], w[k])] == []
