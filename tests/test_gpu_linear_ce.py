"""Softmax cross entropy at the output head (rfq_linear_ce) and its gradients against the
definition in float64.

Tolerances, by arithmetic:
* a logit is an fp32 sum of exact products: off by at most z_tol = 1e-5 * max_tv sum_k |h w|
  (the bound the GEMM's tests use);
* lse: z_tol, plus the sum of exponentials (2^-22 from the exponential, chains of at most
  32 + 5 + 64 + 32 fp32 additions: 1e-5 relative), plus one fp32 rounding of lse and the
  fp32 rounding of max * log2 e and of each exponent (4 * 2^-24 |lse|);
* loss: lse's and the label's logit's;
* dz = g (p - [v = y]) is rounded once to bf16 (2^-8 relative) and p is off by the relative
  error of lse and z; so dh is off by at most (2^-8 + p_tol + 1e-5) sum_v (|g| (p + [v = y])) |w|
  plus its own rounding 2^-8 |dh|, and dw the same with |h|.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

IGNORE = -100


def make(T, D, V, seed=0, std=1.5, ignore_share=0.1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    w = (torch.randn((V, D), generator=g, device="cuda") * (std / D ** 0.5)).bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    drop = torch.rand((T,), generator=g, device="cuda") < ignore_share
    drop[0] = False
    labels = torch.where(drop, torch.full_like(labels, IGNORE), labels)
    dloss = torch.rand((T,), generator=g, device="cuda") + 0.1
    return h, w, labels, dloss


def reference(h, w, labels, dloss, ignore=IGNORE):
    h, w = h.double(), w.double()
    z = h @ w.T
    z_tol = 1e-5 * float((h.abs() @ w.abs().T).max())
    lse = torch.logsumexp(z, 1)
    counted = labels != ignore
    at = torch.where(counted, labels, 0)
    loss = torch.where(counted, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    p = torch.exp(z - lse[:, None])
    onehot = torch.zeros_like(p).scatter_(1, at[:, None], 1.0)
    g = torch.where(counted, dloss.double(), 0.0)[:, None]
    dz = g * (p - onehot)
    size = g.abs() * (p + onehot)
    lse_tol = z_tol + 1e-5 + 4 * 2.0 ** -24 * lse.abs()
    p_tol = float((lse_tol + z_tol).max()) + 1e-6
    rel = 2.0 ** -8 + p_tol + 1e-5
    dh, dw = dz @ w, dz.T @ h
    return {"lse": (lse, lse_tol), "loss": (loss, lse_tol + z_tol),
            "dh": (dh, rel * (size @ w.abs()) + 2.0 ** -8 * dh.abs()),
            "dw": (dw, rel * (size.T @ h.abs()) + 2.0 ** -8 * dw.abs())}


def check(name, got, want):
    ref, tol = want
    err = (got.double() - ref).abs()
    over = (err - tol).max()
    assert torch.isfinite(got.float()).all(), f"{name}: not finite"
    assert float(over) <= 0, f"{name}: off by {float(err.max()):.3e}, {float(over):.3e} over the bound"


SHAPES = [(1, 8, 1), (1, 64, 2), (2, 72, 255), (3, 1024, 5003), (127, 200, 256), (128, 64, 257), (129, 128, 1000),
          (256, 136, 999), (300, 512, 2049), (513, 256, 777), (700, 2048, 300), (64, 4096, 12289)]


@pytest.mark.parametrize("T,D,V", SHAPES)
def test_forward_and_gradients(rfq, T, D, V):
    h, w, labels, dloss = make(T, D, V, seed=T + V)
    want = reference(h, w, labels, dloss)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    torch.cuda.synchronize()
    rfq.check_device_error()
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])


def test_several_pieces_of_the_vocabulary(rfq):
    T, D, V = 16384, 64, 20001   # 16384 rows cut this vocabulary into pieces
    h, w, labels, dloss = make(T, D, V, seed=5)
    want = reference(h, w, labels, dloss)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])


def test_more_rows_than_one_forward_pass(rfq):
    T, D, V = 33000, 16, 300
    h, w, labels, dloss = make(T, D, V, seed=6)
    want = reference(h, w, labels, dloss)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])


@pytest.mark.parametrize("want_dh,want_dw", [(True, False), (False, True)])
def test_one_gradient_alone_is_the_same_bits(rfq, want_dh, want_dw):
    h, w, labels, dloss = make(200, 128, 1500, seed=9)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    both = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    one = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss, want_dh, want_dw)
    for a, b in zip(both, one):
        assert b is None or torch.equal(a, b)
    assert (one[0] is not None) == want_dh and (one[1] is not None) == want_dw


def test_peaked_rows_and_large_logits(rfq):
    """Logits of a few hundred, probabilities that underflow, labels that are certain."""
    h, w, labels, dloss = make(150, 256, 600, seed=3, std=40.0)
    h[::3] += 0.5 * w[labels.clamp(min=0)][::3]
    want = reference(h, w, labels, dloss)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])


def test_every_row_ignored(rfq):
    h, w, labels, dloss = make(130, 64, 300)
    labels.fill_(IGNORE)
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, torch.full_like(dloss, float("nan")))
    assert not loss.any() and torch.isfinite(lse).all()
    assert not dh.any() and not dw.any()


def test_ignored_rows_may_hold_anything(rfq):
    h, w, labels, dloss = make(140, 64, 300, seed=2)
    labels[5] = IGNORE
    base = rfq.linear_ce_alloc(h, w, labels)
    grads = rfq.linear_ce_backward_alloc(h, w, labels, base[1], dloss)
    dloss2 = dloss.clone()
    dloss2[5] = float("inf")
    again = rfq.linear_ce_backward_alloc(h, w, labels, base[1], dloss2)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_ignore_index_inside_the_vocabulary(rfq):
    h, w, labels, dloss = make(140, 64, 300, seed=4, ignore_share=0)
    labels[::4] = 7
    want = reference(h, w, labels, dloss, ignore=7)
    loss, lse = rfq.linear_ce_alloc(h, w, labels, ignore_index=7)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss, ignore_index=7)
    assert not loss[::4].any()
    for name, got in (("lse", lse), ("loss", loss), ("dh", dh), ("dw", dw)):
        check(name, got, want[name])


@pytest.mark.parametrize("bad", [300, -1, 1 << 40])
def test_label_outside_the_vocabulary_is_loud(rfq, bad):
    h, w, labels, dloss = make(140, 64, 300, seed=4, ignore_share=0)
    labels[9] = bad
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, _ = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss, want_dw=False)
    keep = torch.arange(140, device="cuda") != 9
    assert torch.isnan(loss[9]) and torch.isnan(dh[9].float()).all()
    assert torch.isfinite(loss[keep]).all() and torch.isfinite(lse).all() and torch.isfinite(dh[keep].float()).all()


def test_non_finite_rows_stay_in_their_rows(rfq):
    h, w, labels, dloss = make(140, 64, 300, seed=8, ignore_share=0)
    want = reference(h, w, labels, dloss)
    h[3, 0] = float("nan")
    h[77, 1] = float("inf")
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[[3, 77]] = False
    assert not torch.isfinite(loss[~keep]).any()
    ref, tol = want["loss"]
    assert ((loss.double() - ref).abs() <= tol)[keep].all()


def test_zero_and_uneven_dloss(rfq):
    h, w, labels, dloss = make(260, 64, 500, seed=11)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, torch.zeros_like(dloss))
    assert not dh.any() and not dw.any()
    dloss = dloss * torch.logspace(-6, 3, 260, device="cuda")
    dloss[::5] = 0
    dloss[1::5] *= -1
    want = reference(h, w, labels, dloss)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    check("dh", dh, want["dh"])
    check("dw", dw, want["dw"])


def test_gradients_are_the_differences_of_the_loss(rfq):
    """Central differences of the float64 loss along a direction, against the returned gradients: the step's
    third-order error is far below the bf16 rounding of dz and of the gradient."""
    h, w, labels, dloss = make(64, 128, 400, seed=13)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    want = reference(h, w, labels, dloss)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    uh = torch.randn(h.shape, generator=g, device="cuda", dtype=torch.float64)
    uw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)

    def total(eps_h, eps_w):
        z = (h.double() + eps_h * uh) @ (w.double() + eps_w * uw).T
        loss = torch.logsumexp(z, 1) - z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
        return float((loss * torch.where(labels != IGNORE, dloss.double(), 0.0)).sum())

    e = 1e-5
    for got, u, diff, name in ((dh, uh, (total(e, 0) - total(-e, 0)) / (2 * e), "dh"),
                               (dw, uw, (total(0, e) - total(0, -e)) / (2 * e), "dw")):
        tol = float((want[name][1] * u.abs()).sum()) + 1e-6 * abs(diff) + 1e-5
        assert abs(float((got.double() * u).sum()) - diff) <= tol


def test_repeats_bit_for_bit_and_leaves_its_inputs(rfq):
    h, w, labels, dloss = make(513, 520, 3001, seed=21)
    kept = [t.clone() for t in (h, w, labels, dloss)]
    first = rfq.linear_ce_alloc(h, w, labels)
    grads = rfq.linear_ce_backward_alloc(h, w, labels, first[1], dloss)
    for _ in range(5):
        again = rfq.linear_ce_alloc(h, w, labels)
        g2 = rfq.linear_ce_backward_alloc(h, w, labels, again[1], dloss)
        assert all(torch.equal(a, b) for a, b in zip(first + grads, again + g2))
    assert all(torch.equal(a, b) for a, b in zip(kept, (h, w, labels, dloss)))


def test_nothing_outside_the_outputs_is_written(rfq):
    T, D, V = 130, 72, 301
    h, w, labels, dloss = make(T, D, V, seed=22)
    pad = 64

    def fenced(n, dtype):
        t = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device="cuda")
        return t, t[pad:pad + n]

    loss_f, loss = fenced(T, torch.float32)
    lse_f, lse = fenced(T, torch.float32)
    dh_f, dh = fenced(T * D, torch.bfloat16)
    dw_f, dw = fenced(V * D, torch.bfloat16)
    need = rfq.linear_ce_workspace_bytes(T, D, V, True, True)
    ws_f = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")
    ws = ws_f[256:256 + need]
    rfq.linear_ce(h, w, labels, loss, lse, ws)
    rfq.linear_ce_backward(h, w, labels, lse, dloss, dh.view(T, D), dw.view(V, D), ws)
    torch.cuda.synchronize()
    for f in (loss_f, lse_f, dh_f, dw_f):
        assert (f[:pad] == 7).all() and (f[-pad:] == 7).all()
    assert (ws_f[:256] == 165).all() and (ws_f[256 + need:] == 165).all()
    want = reference(h, w, labels, dloss)
    check("dw", dw.view(V, D), want["dw"])


def test_captured_graph_follows_its_inputs(rfq):
    T, D, V = 300, 128, 1200
    h, w, labels, dloss = make(T, D, V, seed=30)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(rfq.linear_ce_workspace_bytes(T, D, V, True, True), dtype=torch.uint8, device="cuda")

    def step():
        rfq.linear_ce(h, w, labels, loss, lse, ws)
        rfq.linear_ce_backward(h, w, labels, lse, dloss, dh, dw, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (31, 32):
        for dst, src in zip((h, w, labels, dloss), make(T, D, V, seed=seed)):
            dst.copy_(src)
        graph.replay()
        got = [t.clone() for t in (loss, lse, dh, dw)]
        want = reference(h, w, labels, dloss)
        for name, t in zip(("loss", "lse", "dh", "dw"), got):
            check(name, t, want[name])


def test_another_stream(rfq):
    h, w, labels, dloss = make(300, 128, 1200, seed=40)
    base = rfq.linear_ce_alloc(h, w, labels)
    grads = rfq.linear_ce_backward_alloc(h, w, labels, base[1], dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (side, side.cuda_stream):
        o = rfq.linear_ce_alloc(h, w, labels, stream=stream)
        outs.append(o + rfq.linear_ce_backward_alloc(h, w, labels, o[1], dloss, stream=stream))
    side.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(base + grads, o))


def test_offsets_past_32_bits(rfq):
    """A head of more than 2^31 elements: the last entries of the vocabulary and the last rows of its gradient."""
    T, D, V = 3, 2048, (1 << 20) + 1001
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    h = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    w = torch.empty((V, D), dtype=torch.bfloat16, device="cuda")
    for part in w.split(1 << 16):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * (1.5 / D ** 0.5))
    labels = torch.tensor([V - 1, 5, V - 700], device="cuda")
    dloss = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    z = torch.cat([h.double() @ part.double().T for part in w.split(1 << 16)], 1)
    lse64 = torch.logsumexp(z, 1)
    z_tol = 1e-5 * float((h.double().abs() @ w[-1000:].double().abs().T).max()) * 1.5
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    tol = z_tol + 1e-5 + 4 * 2.0 ** -24 * lse64.abs()
    assert ((lse.double() - lse64).abs() <= tol).all()
    assert ((loss.double() - (lse64 - z.gather(1, labels[:, None])[:, 0])).abs() <= tol + z_tol).all()
    _, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss, want_dh=False)
    p = torch.exp(z[:, -1000:] - lse64[:, None])
    onehot = torch.zeros_like(p)
    onehot[0, 999] = 1.0
    onehot[2, 300] = 1.0
    gd = dloss.double()[:, None]
    want = (gd * (p - onehot)).T @ h.double()
    bound = (2.0 ** -8 + 2 * float(tol.max()) + 1e-5) * ((gd * (p + onehot)).T @ h.double().abs()) + 2.0 ** -8 * want.abs()
    assert ((dw[-1000:].double() - want).abs() <= bound).all()


def test_no_rows(rfq):
    h = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.randn((100, 64), device="cuda").bfloat16()
    labels, z = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = rfq.linear_ce_alloc(h, w, labels)
    assert loss.shape == (0,) and lse.shape == (0,)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, z, z)
    assert dh.shape == (0, 64) and not dw.any()


def test_binding_refuses_what_the_kernel_cannot_read(rfq):
    h, w, labels, dloss = make(16, 64, 100)
    loss, lse = torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
    ws = torch.empty(rfq.linear_ce_workspace_bytes(16, 64, 100), dtype=torch.uint8, device="cuda")
    for args in [(h.float(), w, labels, loss, lse, ws), (h, w.half(), labels, loss, lse, ws),
                 (h, w, labels.int(), loss, lse, ws), (h, w, labels[:8], loss, lse, ws),
                 (torch.empty((64, 16), dtype=torch.bfloat16, device="cuda").T, w, labels, loss, lse, ws),
                 (h, w, labels, loss.double(), lse, ws), (h, w, labels, loss, lse.cpu(), ws),
                 (h, w, labels, loss, lse, ws.cpu()), (h.cpu(), w, labels, loss, lse, ws)]:
        with pytest.raises(rfq.RFQError, match="INVALID_ARG|want a|workspace is") as e:
            rfq.linear_ce(*args)
        assert e.value.status == 1
    with pytest.raises(rfq.RFQError) as e:
        rfq.linear_ce(h, w, labels, loss, lse, ws[:100])
    assert e.value.status == 7


@pytest.mark.parametrize("T", [1, 2, 16])
def test_gradients_of_few_rows_are_rounded_once(rfq, T):
    """Up to 16 rows the softmax's gradient enters the products with 16 bits: what is left is the rounding of the
    outputs (2^-8 of each entry) and, of the terms that were summed, 2^-14 (2^-17 from the two terms, below 2^-16 from
    exponentials, the label's p - 1 and fp32 sums of up to 300 terms)."""
    D, V = 72, 300
    h, w, labels, dloss = make(T, D, V, seed=40 + T, ignore_share=0)
    _, lse = rfq.linear_ce_alloc(h, w, labels)
    dh, dw = rfq.linear_ce_backward_alloc(h, w, labels, lse, dloss)
    h64, w64 = h.double(), w.double()
    z = h64 @ w64.t()
    dz = (torch.softmax(z, 1) - torch.nn.functional.one_hot(labels, V)) * dloss.double()[:, None]
    for got, want, terms in ((dh, dz @ w64, dz.abs() @ w64.abs()), (dw, dz.t() @ h64, dz.abs().t() @ h64.abs())):
        assert ((got.double() - want).abs() <= 2.0**-8 * want.abs() + 2.0**-14 * terms).all()


@pytest.mark.parametrize("T,D,V", [(3, 40008, 300), (16, 65536, 72), (200, 65536, 264), (16, 8, 20001), (17, 8, 20001)])
def test_more_tiles_than_units(rfq, T, D, V):
    """Hidden states wider than a round of tiles, and both sides of the border between one and two terms of dz."""
    test_forward_and_gradients(rfq, T, D, V)
