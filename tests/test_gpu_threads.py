"""Calls from several host threads at once: the library is thread-safe, so calls of other sizes, each with a stream, tensors and a
workspace of its own, do not disturb one another."""
import threading

import pytest
import torch

from tests.test_gpu_linear_ce import make as make_head
from tests.test_gpu_lora import BF16, F32, make

pytestmark = pytest.mark.gpu


def adapters(rfq, shape, dtype, stream, rounds, wrong, barrier):
    try:
        torch.cuda.set_device(0)
        with torch.cuda.stream(stream):
            c = make(*shape, "runs", seed=shape[3], dtype=dtype)
            M, K, N, r, n = shape
            y, hidden = torch.empty_like(c["base"]), torch.empty((M, r), device="cuda")
            dx, da, db = torch.empty_like(c["dx_base"]), torch.empty_like(c["a"], dtype=dtype), torch.empty_like(c["b"], dtype=dtype)
            ws = torch.empty(rfq.lora_workspace_bytes(M, K, N, r, n, backward=True), dtype=torch.uint8, device="cuda")
            stream.synchronize()
            first = None
            barrier.wait()
            for i in range(rounds):
                rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], y, ws, base=c["base"], hidden=hidden)
                rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], hidden, ws, dx=dx, dx_base=c["dx_base"], da=da, db=db)
                if i == 0 or i == rounds - 1:
                    stream.synchronize()
                    now = [t.clone() for t in (y, hidden, dx, da, db)]
                    if first is None:
                        first = now
                    elif not all(torch.equal(a, b) for a, b in zip(first, now)):
                        wrong.append((shape, "results differ"))
            stream.synchronize()
    except Exception as e:   # noqa: BLE001 (reported by the test)
        wrong.append((shape, repr(e)))
        barrier.abort()


# Short batches of two ranks that share a kernel, long ones of two ranks, and both
@pytest.mark.parametrize("shapes", [[(40, 264, 312, 72, 3), (40, 264, 312, 128, 3)], [(300, 4104, 4104, 24, 2), (300, 4104, 4104, 128, 2)],
                                    [(40, 264, 312, 8, 3), (300, 4104, 4104, 64, 2), (40, 264, 312, 128, 3), (1201, 1032, 5128, 40, 3)]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_adapters_of_other_ranks_at_once(rfq, shapes, dtype):
    wrong, barrier = [], threading.Barrier(len(shapes))
    threads = [threading.Thread(target=adapters, args=(rfq, s, dtype, torch.cuda.Stream(), 300, wrong, barrier)) for s in shapes]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads)
    assert wrong == []
    torch.cuda.synchronize()


@pytest.mark.parametrize("r", [8, 32, 56])
def test_long_adapter_batches_beside_short_projections(rfq, r):
    """The adapters' shrink and the short-batch GEMM both run in clusters and hold tensor memory; on two streams at once they must
    not wait for one another (a CTA of the one never shares an SM with one of the other)."""
    M, K, N, n = 4096, 4096, 2048, 3
    c = make(M, K, N, r, n, "runs", seed=r)
    g = torch.Generator(device="cuda")
    g.manual_seed(r)
    qw = rfq.quantize_weight_alloc((torch.randn((4096, 4096), generator=g, device="cuda") * 0.02).bfloat16())
    xs = [torch.randn((rows, 4096), generator=g, device="cuda").bfloat16() for rows in (40, 64, 100)]
    want_y = [rfq.linear_alloc(x, qw, use_residual=False) for x in xs]
    want = rfq.lora_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], base=c["base"], want_hidden=True)
    want_b = rfq.lora_backward_alloc(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], want[1], dx_base=c["dx_base"], want_da=False, want_db=False)
    y, hidden, dx = torch.empty_like(c["base"]), torch.empty_like(want[1]), torch.empty_like(c["dx_base"])
    ws = torch.empty(rfq.lora_workspace_bytes(M, K, N, r, n, backward=True), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in want_y]
    ws_y = [torch.empty(rfq.linear_workspace_bytes(x.shape[0], 4096), dtype=torch.uint8, device="cuda") for x in xs]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(60):
        rfq.lora(c["x"], c["a"], c["b"], c["scale"], c["ids"], y, ws, base=c["base"], hidden=hidden, stream=a)
        rfq.lora_backward(c["x"], c["a"], c["b"], c["scale"], c["ids"], c["dy"], hidden, ws, dx=dx, dx_base=c["dx_base"], stream=a)
        for _ in range(4):
            for x, out, w in zip(xs, outs, ws_y):
                rfq.linear(x, qw.codes, qw.scales, 4096, out, w, use_residual=False, stream=b)
    torch.cuda.synchronize()
    rfq.check_device_error()
    assert torch.equal(y, want[0]) and torch.equal(hidden, want[1]) and torch.equal(dx, want_b[0])
    assert all(torch.equal(p, q) for p, q in zip(outs, want_y))


def head(rfq, shape, stream, rounds, wrong, barrier):
    try:
        torch.cuda.set_device(0)
        with torch.cuda.stream(stream):
            T, D, V = shape
            h, w, labels, dloss = make_head(T, D, V, seed=T)
            loss, lse, dh, dw = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(h), torch.empty_like(w)
            ws = torch.empty(rfq.linear_ce_workspace_bytes(T, D, V, True, True), dtype=torch.uint8, device="cuda")
            grads = [torch.empty_like(dh), torch.empty_like(dw)]
            norm, clip_ws = torch.empty(1, device="cuda"), torch.empty(rfq.grad_clip_workspace_bytes(2), dtype=torch.uint8, device="cuda")
            stream.synchronize()
            first = None
            barrier.wait()
            for i in range(rounds):
                rfq.linear_ce(h, w, labels, loss, lse, ws)
                rfq.linear_ce_backward(h, w, labels, lse, dloss, dh, dw, ws)
                rfq.grad_clip([dh, dw], 0.5, norm, clip_ws, outs=grads)
                if i == 0 or i == rounds - 1:
                    stream.synchronize()
                    now = [t.clone() for t in (loss, lse, dh, dw, norm, *grads)]
                    if first is None:
                        first = now
                    elif not all(torch.equal(a, b) for a, b in zip(first, now)):
                        wrong.append((shape, "results differ"))
            stream.synchronize()
    except Exception as e:   # noqa: BLE001 (reported by the test)
        wrong.append((shape, repr(e)))
        barrier.abort()


def test_every_operator_at_once(rfq):
    """Heads of few and many rows with their gradients clipped, adapters of short and long batches: a thread and a stream each."""
    heads, batches = [(9, 264, 3000), (100, 520, 20000), (600, 256, 5000)], [(40, 264, 312, 72, 3), (1201, 1032, 5128, 40, 3)]
    wrong, barrier = [], threading.Barrier(len(heads) + len(batches))
    threads = [threading.Thread(target=head, args=(rfq, s, torch.cuda.Stream(), 100, wrong, barrier)) for s in heads]
    threads += [threading.Thread(target=adapters, args=(rfq, s, BF16, torch.cuda.Stream(), 100, wrong, barrier)) for s in batches]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads)
    assert wrong == []
    torch.cuda.synchronize()
    rfq.check_device_error()
