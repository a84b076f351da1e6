"""One fine-tuning step of low-rank adapters on a frozen MXFP4 projection, made of the library's calls:

    y      = rfq_linear_lora(x)                 frozen W, trained adapters
    loss   = rfq_linear_ce(y, head)             frozen head
    dy     = rfq_linear_ce_backward             gradient of the hidden states alone
    dx     = rfq_linear_dgrad(dy) ; rfq_lora_backward adds the adapters' share; dA, dB
    norm   = rfq_grad_clip([dA, dB])

Every stage is checked against float64 on what the stage before it gave, so that each tolerance is
that stage's own (they are derived in the tests of the single calls); then the whole step is captured
and replayed, bit for bit the same.
"""
import pytest
import torch

from tests.test_gpu_grad_clip import check_clip
from tests.test_gpu_linear_ce import check as check_ce
from tests.test_gpu_linear_ce import reference as ce_reference
from tests.test_gpu_lora import check as check_lora
from tests.test_gpu_lora import reference as lora_reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Step:
    def __init__(self, rfq, M, K, N, V, r, n, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        self.rfq, self.M, self.K, self.N = rfq, M, K, N
        self.x = normal(M, K).bfloat16()
        w = normal(N, K, std=K ** -0.5).bfloat16()
        self.qw = rfq.quantize_weight_alloc(w)
        self.qwt = rfq.quantize_mxfp4_t_alloc(w, residual=False)      # W^T along N, for dgrad
        self.a, self.b = normal(n, r, K, std=K ** -0.5).bfloat16(), normal(n, N, r, std=r ** -0.5).bfloat16()
        self.scale = torch.full((n,), 0.5, device="cuda")
        self.ids = torch.sort(torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)).values
        self.head = normal(V, N, std=2 * N ** -0.5).bfloat16()
        self.labels = torch.randint(0, V, (M,), generator=g, device="cuda")
        self.labels[::7] = -100
        counted = self.labels != -100
        self.dloss = counted.float() / counted.sum()
        e = dict(device="cuda")
        self.y, self.dy = torch.empty((M, N), dtype=BF16, **e), torch.empty((M, N), dtype=BF16, **e)
        self.loss, self.lse = torch.empty(M, **e), torch.empty(M, **e)
        self.hidden, self.dx = torch.empty((M, r), **e), torch.empty((M, K), dtype=BF16, **e)
        self.dx_frozen = torch.empty_like(self.dx)
        self.da, self.db = torch.empty_like(self.a), torch.empty_like(self.b)
        self.clipped = [torch.empty_like(self.da), torch.empty_like(self.db)]
        self.norm = torch.empty(1, **e)
        u8 = dict(dtype=torch.uint8, **e)
        # one workspace for every call of the step: they follow one another on one stream
        self.ws = torch.empty(max(rfq.linear_lora_workspace_bytes(M, K, N, r, n), rfq.linear_ce_workspace_bytes(M, N, V, True, False),
                                  rfq.linear_workspace_bytes(M, N), rfq.lora_workspace_bytes(M, K, N, r, n, True), rfq.grad_clip_workspace_bytes(2)), **u8)
        self.max_norm = 1e-3

    def run(self):
        rfq, ws = self.rfq, self.ws
        rfq.linear_lora(self.x, self.qw.codes, self.qw.scales, self.N, self.a, self.b, self.scale, self.ids, self.y, ws, hidden=self.hidden)
        rfq.linear_ce(self.y, self.head, self.labels, self.loss, self.lse, ws)
        rfq.linear_ce_backward(self.y, self.head, self.labels, self.lse, self.dloss, self.dy, None, ws)
        rfq.linear_dgrad(self.dy, self.qwt.codes, self.qwt.scales, self.K, self.dx_frozen, ws)
        rfq.lora_backward(self.x, self.a, self.b, self.scale, self.ids, self.dy, self.hidden, ws, dx=self.dx, dx_base=self.dx_frozen, da=self.da,
                          db=self.db)
        rfq.grad_clip([self.da, self.db], self.max_norm, self.norm, ws, outs=self.clipped)

    def results(self):
        return [t.clone() for t in (self.y, self.loss, self.lse, self.dy, self.dx_frozen, self.dx, self.hidden, self.da, self.db, self.norm, *self.clipped)]


@pytest.mark.parametrize("M,K,N,V,r,n", [(24, 256, 512, 1000, 8, 3), (300, 512, 256, 3001, 16, 4), (1000, 1024, 512, 2000, 64, 2)])
def test_step(rfq, M, K, N, V, r, n):
    s = Step(rfq, M, K, N, V, r, n, seed=M)
    s.run()
    torch.cuda.synchronize()
    rfq.check_device_error()
    base = rfq.linear_alloc(s.x, s.qw)
    c = {"x": s.x, "a": s.a, "b": s.b, "scale": s.scale, "ids": s.ids, "base": base, "dy": s.dy, "dx_base": s.dx_frozen}
    want = lora_reference(c)
    for name, t in (("y", s.y), ("hidden", s.hidden), ("dx", s.dx), ("da", s.da), ("db", s.db)):
        check_lora(name, t, want[name])
    want = ce_reference(s.y, s.head, s.labels, s.dloss)
    for name, t in (("loss", s.loss), ("lse", s.lse), ("dh", s.dy)):
        check_ce(name, t, want[name])
    assert torch.equal(s.dx_frozen, rfq.linear_dgrad_alloc(s.dy, s.qwt))
    check_clip([s.da, s.db], s.clipped, s.norm, s.max_norm)
    assert float(s.norm) > s.max_norm   # it does clip

    first = s.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t in (s.y, s.dy, s.dx, s.da, s.db, s.norm, s.hidden):
        t.fill_(float("nan"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, s.results()))


def test_two_steps_at_once(rfq):
    """Two steps on two streams, each with buffers of its own, give what each gives alone."""
    steps = [Step(rfq, 300, 512, 256, 3001, 16, 4, seed=i) for i in (1, 2)]
    alone = []
    for s in steps:
        s.run()
        alone.append(s.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, want in zip(steps, alone):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), want))
    rfq.check_device_error()
