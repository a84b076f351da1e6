"""Calls from several host threads at once: the library is thread-safe, so calls of other sizes, each with a stream, tensors and a
workspace of its own, do not disturb one another."""
import threading

import pytest
import torch

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
