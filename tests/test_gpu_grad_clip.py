"""Global gradient norm and clipping (rfq_grad_norm, rfq_grad_clip) against float64.

Tolerances, by arithmetic: 32 squares are summed in fp32 (at most 33 roundings of 2^-24 in a sum
of positive terms, halved by the square root), everything after in fp64, and the norm is rounded
once: 18 * 2^-24 relative.  The factor adds two more roundings (the sum with 1e-6, the division)
and the product one of its own: 22 * 2^-24 relative, plus 2^-8 where the result is bf16.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
NORM_TOL, OUT_TOL = 18 * 2.0 ** -24, 22 * 2.0 ** -24


def make(sizes, seed=0, std=1e-2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(t) for n, t in sizes]


def norm64(grads):
    return float(torch.stack([t.double().square().sum() for t in grads] + [torch.zeros((), dtype=torch.float64, device="cuda")]).sum().sqrt())


def check_clip(grads, outs, norm, max_norm):
    want = norm64(grads)
    assert abs(float(norm) - want) <= NORM_TOL * want
    c = min(1.0, max_norm / (want + 1e-6))
    for x, y in zip(grads, outs):
        ref = x.double() * c
        tol = ref.abs() * (OUT_TOL + (2.0 ** -8 if x.dtype == BF16 else 0.0))
        tol = tol + (2.0 ** -134 if x.dtype == BF16 else 2.0 ** -149)   # subnormal results
        assert y.dtype == x.dtype and ((y.double() - ref).abs() <= tol).all()


LISTS = [[(1, F32)], [(1, BF16)], [(7, BF16), (8, F32), (9, BF16)], [(8191, BF16), (8192, BF16), (8193, F32), (1, BF16)],
         [(100000, BF16), (3, F32), (70001, F32)], [(n, (BF16, F32)[n % 2]) for n in range(1, 1200)], [(5_000_011, BF16), (4_000_000, F32)]]


@pytest.mark.parametrize("sizes", LISTS, ids=[f"{len(s)}x{s[-1][0]}" for s in LISTS])
@pytest.mark.parametrize("max_norm", [0.05, 1e6, float("inf"), 0.0])
def test_norm_and_clip(rfq, sizes, max_norm):
    grads = make(sizes, seed=len(sizes))
    want = norm64(grads)
    norm = rfq.grad_norm_alloc(grads)
    assert abs(float(norm) - want) <= NORM_TOL * want
    kept = [t.clone() for t in grads]
    outs = [torch.full_like(t, 9.0) for t in grads]
    ws = torch.empty(rfq.grad_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device="cuda")
    norm2 = torch.empty(1, device="cuda")
    rfq.grad_clip(grads, max_norm, norm2, ws, outs=outs)
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(grads, kept))
    check_clip(kept, outs, norm2, max_norm)
    norm3 = rfq.grad_clip_alloc(grads, max_norm)
    assert torch.equal(norm, norm3) and all(torch.equal(a, b) for a, b in zip(grads, outs))


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_unaligned_views(rfq, offset):
    flats = [torch.full((20011 + 64,), 7.0, dtype=t, device="cuda") for t in (BF16, F32)]
    grads = []
    for f, src in zip(flats, make([(20011, BF16), (20011, F32)], seed=3)):
        v = f[offset:offset + 20011]
        v.copy_(src)
        grads.append(v)
    kept = [t.clone() for t in grads]
    norm = rfq.grad_clip_alloc(grads, 0.1)
    check_clip(kept, grads, norm, 0.1)
    for f in flats:
        assert (f[:offset] == 7).all() and (f[offset + 20011:] == 7).all()


def test_nothing_past_an_output_is_written(rfq):
    grads = make([(8193, BF16), (8195, F32)], seed=4)
    flats = [torch.full((t.numel() + 64,), 7.0, dtype=t.dtype, device="cuda") for t in grads]
    outs = [f[:t.numel()] for f, t in zip(flats, grads)]
    norm = torch.empty(1, device="cuda")
    ws_f = torch.full((rfq.grad_clip_workspace_bytes(2) + 256,), 165, dtype=torch.uint8, device="cuda")
    rfq.grad_clip(grads, 0.1, norm, ws_f[:-256], outs=outs)
    check_clip(grads, outs, norm, 0.1)
    assert all((f[t.numel():] == 7).all() for f, t in zip(flats, grads)) and (ws_f[-256:] == 165).all()


@pytest.mark.parametrize("std", [1e-30, 1e-22, 1e-16, 1e16, 1e19, 3e30])
def test_the_norm_neither_overflows_nor_underflows_on_its_way(rfq, std):
    grads = make([(8192, F32), (1000, F32), (9000, BF16)], seed=5, std=std)
    want = norm64(grads)
    norm = rfq.grad_norm_alloc(grads)
    assert abs(float(norm) - want) <= NORM_TOL * want


def test_empty_list_and_empty_tensors(rfq):
    assert float(rfq.grad_norm_alloc([])) == 0.0
    assert float(rfq.grad_clip_alloc([], 1.0)) == 0.0
    grads = [torch.empty(0, device="cuda"), torch.tensor([3.0, 4.0], device="cuda"), torch.empty((0, 5), dtype=BF16, device="cuda")]
    assert float(rfq.grad_clip_alloc(grads, 1.0)) == 5.0
    assert float(rfq.grad_norm_alloc([torch.zeros(10000, device="cuda")])) == 0.0


@pytest.mark.parametrize("bad,factor", [(float("inf"), 0.0), (float("nan"), float("nan"))])
def test_values_that_are_not_finite(rfq, bad, factor):
    grads = make([(9000, F32), (100, BF16)], seed=6)
    grads[0][8500] = bad
    norm = rfq.grad_clip_alloc(grads, 1.0)
    assert not torch.isfinite(norm).any()
    if factor == 0.0:
        assert torch.isnan(grads[0][8500]) and not grads[1].any()
    else:
        assert torch.isnan(grads[0]).all() and torch.isnan(grads[1]).all()


def test_a_factor_of_one_leaves_the_bits(rfq):
    grads = make([(9000, F32), (100, BF16)], seed=7)
    kept = [t.clone() for t in grads]
    rfq.grad_clip_alloc(grads, 100.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_repeats_bit_for_bit(rfq):
    grads = make([(3_000_001, BF16), (777, F32), (2_000_000, F32)], seed=8)
    first = rfq.grad_norm_alloc(grads)
    assert all(torch.equal(first, rfq.grad_norm_alloc(grads)) for _ in range(10))


def test_captured_graph_follows_its_inputs(rfq):
    grads = make([(9000, F32), (600, BF16)] * 300, seed=9)   # more than one table of tensors
    norm = torch.empty(1, device="cuda")
    outs = [torch.empty_like(t) for t in grads]
    ws = torch.empty(rfq.grad_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device="cuda")
    rfq.grad_clip(grads, 0.5, norm, ws, outs=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rfq.grad_clip(grads, 0.5, norm, ws, outs=outs)
    for seed, std in ((10, 1e-2), (11, 1e-6)):
        for dst, src in zip(grads, make([(t.numel(), t.dtype) for t in grads], seed=seed, std=std)):
            dst.copy_(src)
        graph.replay()
        check_clip(grads, outs, norm, 0.5)


def test_another_stream(rfq):
    grads = make([(9000, F32), (600, BF16)], seed=12)
    first = rfq.grad_norm_alloc(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rfq.grad_norm_alloc(grads, stream=side)
    side.synchronize()
    assert torch.equal(first, got)


def test_binding_refuses_what_the_kernel_cannot_read(rfq):
    grads = make([(64, F32), (64, BF16)])
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(rfq.grad_clip_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    for bad in ([grads[0].double()], [grads[0].cpu()], [torch.empty((8, 8), device="cuda").T], [grads[0].half()]):
        with pytest.raises(rfq.RFQError) as e:
            rfq.grad_norm(bad, norm, ws)
        assert e.value.status == 1
    for outs in (grads[:1], [grads[1], grads[0]], [grads[0][:32], grads[1]]):
        with pytest.raises(rfq.RFQError) as e:
            rfq.grad_clip(grads, 1.0, norm, ws, outs=outs)
        assert e.value.status == 1
    for bad in (-1.0, float("nan")):
        with pytest.raises(rfq.RFQError) as e:
            rfq.grad_clip(grads, bad, norm, ws)
        assert e.value.status == 1
    with pytest.raises(rfq.RFQError) as e:
        rfq.grad_norm(grads, norm, ws[:64])
    assert e.value.status == 7
