"""Refusals and sizes of the output-head, adapter and clipping calls on a host without a GPU: every
check comes before a device is touched (no address here is ever dereferenced)."""
import ctypes

import pytest
import torch

import block_scaled_gemm_rfq_b200 as rfq
from block_scaled_gemm_rfq_b200 import build as rfq_build

# The addresses are made up: beside a GPU a call whose arguments pass would be launched on them.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="needs a host without a GPU")

A = 1 << 20   # an aligned address
NO_DEVICE = (4, 5)   # what a call says here once its arguments have passed


@pytest.fixture(scope="module")
def lib():
    rfq_build.build()
    return rfq.load_library()


def vp(v):
    return ctypes.c_void_p(v)


def ce(lib, **k):
    d = dict(h=A, w=A, labels=A, T=16, D=64, V=1000, ignore=-100, loss=A, lse=A, ws=A, bytes=1 << 40)
    d.update(k)
    return lib.rfq_linear_ce(vp(d["h"]), vp(d["w"]), vp(d["labels"]), d["T"], d["D"], d["V"], d["ignore"], vp(d["loss"]), vp(d["lse"]),
                             vp(d["ws"]), d["bytes"], None)


def ce_back(lib, **k):
    d = dict(h=A, w=A, labels=A, lse=A, dloss=A, T=16, D=64, V=1000, ignore=-100, dh=A, dw=A, ws=A, bytes=1 << 40)
    d.update(k)
    return lib.rfq_linear_ce_backward(vp(d["h"]), vp(d["w"]), vp(d["labels"]), vp(d["lse"]), vp(d["dloss"]), d["T"], d["D"], d["V"], d["ignore"],
                                      vp(d["dh"]), vp(d["dw"]), vp(d["ws"]), d["bytes"], None)


@pytest.mark.parametrize("call", [ce, ce_back])
@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), 1), (dict(D=-8), 1), (dict(V=-1), 1), (dict(D=12), 2), (dict(D=0), 2), (dict(V=0), 2), (dict(D=65544), 2),
    (dict(T=(1 << 24) + 1), 2), (dict(V=(1 << 24) + 1), 2), (dict(h=None), 1), (dict(w=None), 1), (dict(labels=None), 1), (dict(lse=None), 1),
    (dict(h=A + 2), 3), (dict(w=A + 8), 3), (dict(labels=A + 4), 3), (dict(lse=A + 2), 3), (dict(ws=None), 7), (dict(bytes=100), 7), (dict(ws=A + 128), 3)])
def test_output_head_refuses(lib, call, bad, status):
    assert call(lib, **bad) == status


def test_output_head_refuses_its_own(lib):
    assert ce(lib, loss=None) == 1 and ce(lib, loss=A + 2) == 3
    assert ce_back(lib, dloss=None) == 1 and ce_back(lib, dh=A + 8) == 3 and ce_back(lib, dw=A + 2) == 3
    assert ce(lib) in NO_DEVICE and ce_back(lib) in NO_DEVICE
    # nothing to do
    assert ce(lib, T=0, h=None, ws=None, bytes=0) == 0
    assert ce_back(lib, dh=None, dw=None) == 0
    assert ce_back(lib, T=0, dw=None, ws=None, bytes=0) == 0
    # a workspace for the forward pass alone is too small for a gradient
    assert ce_back(lib, T=3000, V=50000, bytes=rfq.linear_ce_workspace_bytes(3000, 64, 50000)) == 7


def test_output_head_workspace_sizes(lib):
    f = rfq.linear_ce_workspace_bytes
    assert f(0, 64, 100) == 0 and f(16, 12, 100) == 0 and f(-1, 64, 100) == 0
    assert f(16, 64, 1000) % 256 == 0 and 0 < f(16, 64, 1000) <= f(16, 64, 1000, True, True)
    # bounded: the piece of dz is at most 256 MiB (or 2048 columns), whatever the vocabulary
    assert f(4096, 4096, 1 << 24, True, True) < (256 << 20) + 4096 * 4096 * 4 + (64 << 20) + f(4096, 4096, 1 << 24)
    assert f(1 << 20, 64, 1000) < 300 << 20   # the statistics are those of 32768 rows at a time


def lora(lib, **k):
    d = dict(x=A, M=16, K=64, a=A, b=A, scale=A, ids=A, n=4, r=16, N=72, base=A, y=A, t=1, hidden=A, ws=A, bytes=1 << 40)
    d.update(k)
    return lib.rfq_lora(vp(d["x"]), d["M"], d["K"], vp(d["a"]), vp(d["b"]), vp(d["scale"]), vp(d["ids"]), d["n"], d["r"], d["N"], vp(d["base"]), vp(d["y"]),
                        d["t"], vp(d["hidden"]), vp(d["ws"]), d["bytes"], None)


def lora_back(lib, **k):
    d = dict(x=A, M=16, K=64, a=A, b=A, scale=A, ids=A, n=4, r=16, N=72, dy=A, hidden=A, dx_base=A, y=A, t=1, da=A, db=A, g=1, ws=A, bytes=1 << 40)
    d.update(k)
    return lib.rfq_lora_backward(vp(d["x"]), d["M"], d["K"], vp(d["a"]), vp(d["b"]), vp(d["scale"]), vp(d["ids"]), d["n"], d["r"], d["N"], vp(d["dy"]),
                                 vp(d["hidden"]), vp(d["dx_base"]), vp(d["y"]), d["t"], vp(d["da"]), vp(d["db"]), d["g"], vp(d["ws"]), d["bytes"], None)


def linear_lora(lib, **k):
    d = dict(x=A, M=16, K=64, a=A, b=A, scale=A, ids=A, n=4, r=16, N=72, y=A, t=1, hidden=A, ws=A, bytes=1 << 40)
    d.update(k)
    return lib.rfq_linear_lora(vp(d["x"]), d["M"], d["K"], vp(A), vp(A), d["N"], vp(d["a"]), vp(d["b"]), vp(d["scale"]), vp(d["ids"]), d["n"], d["r"],
                               vp(d["y"]), d["t"], 1, vp(d["hidden"]), vp(d["ws"]), d["bytes"], None)


@pytest.mark.parametrize("call", [lora, lora_back, linear_lora])
@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), 1), (dict(K=-8), 1), (dict(N=-8), 1), (dict(r=-8), 1), (dict(n=-1), 1), (dict(t=7), 1), (dict(K=12), 2), (dict(N=12), 2),
    (dict(r=12), 2), (dict(r=0), 2), (dict(r=136), 2), (dict(n=0), 2), (dict(n=4097), 2), (dict(M=(1 << 24) + 1), 2), (dict(K=0), 2), (dict(N=0), 2),
    (dict(N=(1 << 20) + 8), 2), (dict(a=None), 1), (dict(b=None), 1), (dict(scale=None), 1), (dict(ids=None), 1), (dict(a=A + 8), 3), (dict(b=A + 2), 3),
    (dict(scale=A + 2), 3), (dict(ids=A + 1), 3), (dict(y=A + 8), 3), (dict(hidden=A + 2), 3), (dict(ws=None), 7), (dict(bytes=64), 7), (dict(ws=A + 16), 3)])
def test_adapters_refuse(lib, call, bad, status):
    assert call(lib, **bad) == status


def test_adapters_refuse_their_own(lib):
    assert lora(lib, x=None) == 1 and lora(lib, y=None) == 1 and lora(lib, base=A + 8) == 3
    assert lora(lib, base=None, hidden=None) in NO_DEVICE and lora(lib) in NO_DEVICE
    assert lora_back(lib, dy=None) == 1 and lora_back(lib, dy=A + 2) == 3 and lora_back(lib, g=9) == 1 and lora_back(lib, dx_base=A + 4) == 3
    assert lora_back(lib, x=None) == 1 and lora_back(lib, hidden=None) == 1 and lora_back(lib, da=A + 8) == 3 and lora_back(lib, db=A + 8) == 3
    assert lora_back(lib, x=None, da=None) in NO_DEVICE and lora_back(lib, hidden=None, db=None) in NO_DEVICE and lora_back(lib) in NO_DEVICE
    assert linear_lora(lib, K=40) == 2 and linear_lora(lib) in NO_DEVICE
    # nothing to do
    assert lora(lib, M=0, x=None, ws=None, bytes=0) == 0 and linear_lora(lib, M=0, ws=None, bytes=0) == 0
    assert lora_back(lib, y=None, da=None, db=None) == 0 and lora_back(lib, M=0, da=None, db=None, ws=None, bytes=0) == 0


@pytest.mark.parametrize("M", [1, 16, 64, 65, 300, 5000])
def test_adapter_workspace_sizes(lib, M):
    f = rfq.lora_workspace_bytes
    assert 0 < f(M, 512, 1024, 16, 4) <= f(M, 512, 1024, 16, 4, backward=True)
    assert f(M, 512, 1024, 16, 4) % 256 == 0 and f(0, 512, 1024, 16, 4) == 0 and f(M, 512, 1020, 16, 4) == 0
    assert rfq.linear_lora_workspace_bytes(M, 512, 1024, 16, 4) >= max(f(M, 512, 1024, 16, 4), rfq.linear_workspace_bytes(M, 512))
    assert rfq.linear_lora_workspace_bytes(M, 520, 1024, 16, 4) == 0


def clip(lib, ptrs, numels, types, count=None, outs=None, max_norm=1.0, norm=A, ws=A, size=1 << 30, scale=True):
    P = ctypes.c_void_p * max(1, len(ptrs))
    p, n, t = P(*ptrs), (ctypes.c_int64 * max(1, len(numels)))(*numels), (ctypes.c_int * max(1, len(types)))(*types)
    o = None if outs is None else P(*outs)
    count = len(ptrs) if count is None else count
    if scale:
        return lib.rfq_grad_clip(p, o, n, t, count, max_norm, vp(norm), vp(ws), size, None)
    return lib.rfq_grad_norm(p, n, t, count, vp(norm), vp(ws), size, None)


@pytest.mark.parametrize("scale", [True, False])
def test_clipping_refuses(lib, scale):
    ok = ([A, A + 2], [10, 10], [0, 1])
    assert clip(lib, *ok, scale=scale) in NO_DEVICE
    assert clip(lib, *ok, count=-1, scale=scale) == 1 and clip(lib, *ok, count=(1 << 24) + 1, scale=scale) == 1
    assert clip(lib, [A, None], [10, 10], [0, 1], scale=scale) == 1
    assert clip(lib, [A, None], [10, 0], [0, 1], scale=scale) in NO_DEVICE   # an empty tensor has no address
    assert clip(lib, [A], [-1], [0], scale=scale) == 1 and clip(lib, [A], [5], [2], scale=scale) == 1
    assert clip(lib, [A + 2], [5], [0], scale=scale) == 3 and clip(lib, [A + 1], [5], [1], scale=scale) == 3
    assert clip(lib, [A], [1 << 43], [0], scale=scale) == 2 and clip(lib, [A, A], [1 << 41, 3 << 40], [0, 0], scale=scale) == 2
    assert clip(lib, *ok, norm=None, scale=scale) == 1 and clip(lib, *ok, norm=A + 2, scale=scale) == 3
    assert clip(lib, *ok, ws=None, scale=scale) == 7 and clip(lib, *ok, size=8, scale=scale) == 7 and clip(lib, *ok, ws=A + 8, scale=scale) == 3


def test_clipping_refuses_its_own(lib):
    ok = ([A], [10], [0])
    assert clip(lib, *ok, max_norm=-1.0) == 1 and clip(lib, *ok, max_norm=float("nan")) == 1
    assert clip(lib, *ok, max_norm=float("inf")) in NO_DEVICE
    assert clip(lib, *ok, outs=[None]) == 1 and clip(lib, *ok, outs=[A + 2]) == 3 and clip(lib, *ok, outs=[A]) in NO_DEVICE
    assert rfq.grad_clip_workspace_bytes(-1) == 0 and 0 < rfq.grad_clip_workspace_bytes(0) <= rfq.grad_clip_workspace_bytes(2000)


def test_limits_match_the_header():
    src = open(rfq_build.INCLUDE + "/rfq.h").read()
    assert f"#define RFQ_LORA_MAX_RANK {rfq.LORA_MAX_RANK}\n" in src and f"#define RFQ_LORA_MAX_ADAPTERS {rfq.LORA_MAX_ADAPTERS}\n" in src


@pytest.mark.parametrize("offset", [4, 8])
def test_the_saved_rank_vectors_are_aligned(lib, offset):
    """They are written and read 16 bytes at a time."""
    assert lora(lib, hidden=A + offset) == 3 and lora_back(lib, hidden=A + offset) == 3 and linear_lora(lib, hidden=A + offset) == 3
