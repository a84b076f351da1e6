"""Work units of the training and adapter operators that stand beside the RFQ linear layer.

Three operators, as a fine-tuning or serving program calls them next to ``rfq_linear``:

* ``ce``    the loss at the output head: softmax cross entropy of ``h @ w.T`` against one label a
            row, without ever holding the [tokens, vocabulary] logits, and its gradients;
* ``lora``  low-rank adapters of many requests at once beside a shared projection,
            ``y = base + scale_a * (x @ A_a.T) @ B_a.T`` with the adapter ``a`` chosen row by row,
            and its gradients;
* ``clip``  the global norm of a list of gradients, and the list scaled down to a largest norm.

``run`` makes the framework's calls where ``own`` is true and the plain torch form elsewhere.
"""
import math
import random

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # scoring the handful of tokens of a short continuation; vocabulary of no round size
        {"name": "ce score 8 tokens", "op": "ce", "T": 8, "D": 1024, "V": 32003, "grad": ""},
        # log-probabilities of a long prompt under a large vocabulary
        {"name": "ce score prompt", "op": "ce", "T": 2048, "D": 4096, "V": 131072, "grad": ""},
        # a micro-batch of full training: loss, gradient of the hidden states and of the head
        {"name": "ce train", "op": "ce", "T": 4096, "D": 4096, "V": 32768, "grad": "hw"},
        # adapter training: the head is frozen, only the hidden states get a gradient; ragged sizes
        {"name": "ce train frozen head", "op": "ce", "T": 1000, "D": 2048, "V": 50001, "grad": "h"},
        # one decoding step of 16 requests, each with an adapter of its own
        {"name": "lora decode 16", "op": "lora", "M": 16, "K": 4096, "N": 4096, "r": 16, "n": 16,
         "rows": "mixed", "type": "bf16", "train": False},
        # one decoding step of a large mixed batch, some rows with no adapter
        {"name": "lora decode 256", "op": "lora", "M": 256, "K": 4096, "N": 12288, "r": 32, "n": 48,
         "rows": "mixed", "type": "bf16", "train": False},
        # prompts of several requests, wide feed-forward projection
        {"name": "lora prefill", "op": "lora", "M": 4096, "K": 4096, "N": 12288, "r": 64, "n": 8,
         "rows": "requests", "type": "bf16", "train": False},
        # a training step of one adapter: forward, gradients of x, A and B
        {"name": "lora train", "op": "lora", "M": 16384, "K": 4096, "N": 4096, "r": 16, "n": 1,
         "rows": "requests", "type": "bf16", "train": True},
        # several adapters trained at once, fp32 outputs and gradients, ragged sizes
        {"name": "lora train f32 ragged", "op": "lora", "M": 1111, "K": 5120, "N": 13824, "r": 8, "n": 3,
         "rows": "requests", "type": "f32", "train": True},
        # the gradients of a set of adapters
        {"name": "clip adapters", "op": "clip", "count": 56, "numel": 65536, "type": "bf16", "odd": False},
        # fp32 and bf16 gradients of odd sizes side by side
        {"name": "clip mixed odd", "op": "clip", "count": 37, "numel": 1500001, "type": "mixed", "odd": True},
        # the gradients of a model's projections
        {"name": "clip projections", "op": "clip", "count": 40, "numel": 50331648, "type": "bf16", "odd": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ce", "ce", "lora", "lora", "lora", "clip"])
    if op == "ce":
        T, D, V = _log(rng, 1, 4096), 8 * _log(rng, 8, 640), _log(rng, 300, 131072)
        while T * D * V > 4096 * 4096 * 32768:
            V = max(300, V // 2)
        return {"op": "ce", "T": T, "D": D, "V": V, "grad": rng.choice(["", "h", "w", "hw", "hw"])}
    if op == "lora":
        M, K, N = _log(rng, 1, 16384), 8 * _log(rng, 16, 1728), 8 * _log(rng, 16, 1728)
        r, n = 8 * _log(rng, 1, 16), _log(rng, 1, 64)
        while M * (K + N) > 16384 * 8192:
            M //= 2
        while n * r > 1024:
            n //= 2
        return {"op": "lora", "M": M, "K": K, "N": N, "r": r, "n": n, "rows": rng.choice(["mixed", "requests", "requests"]) if M <= 512 else "requests",
                "type": rng.choice(["bf16", "bf16", "f32"]), "train": rng.random() < 0.5}
    count, numel = _log(rng, 1, 60), _log(rng, 100, 20000000)
    while count * numel > 500000000:
        count = max(1, count // 2)
    return {"op": "clip", "count": count, "numel": numel, "type": rng.choice(["bf16", "f32", "mixed"]), "odd": rng.random() < 0.5}


def _clip_sizes(case):
    """[(type, elements)]: the list of tensors of a clip case, from the case alone."""
    rng = random.Random(case["count"] * 1000003 + case["numel"])
    got = []
    for i in range(case["count"]):
        n = max(1, case["numel"] // rng.choice([1, 1, 1, 4, 16, 256]))
        if not case["odd"]:
            n = (n + 63) // 64 * 64
        got.append((("bf16", "f32")[i % 2] if case["type"] == "mixed" else case["type"], n))
    return got


def work(case):
    if case["op"] == "ce":
        T, D, V, g = case["T"], case["D"], case["V"], case["grad"]
        b = 2 * (T * D + V * D) + 8 * T + 8 * T + (4 * T + 2 * T * D * ("h" in g) + 2 * V * D * ("w" in g) if g else 0)
        return {"bytes": b, "flops": 2 * T * D * V * (1 + len(g))}
    if case["op"] == "lora":
        M, K, N, r, n = case["M"], case["K"], case["N"], case["r"], min(case["n"], case["M"])
        e = 2 if case["type"] == "bf16" else 4
        b, f = 2 * M * K + 2 * n * r * (K + N) + 4 * M + 2 * e * M * N, 2 * M * r * (K + N)
        if case["train"]:
            # dy and the base of dx read, dx and the two adapter gradients written
            b += 2 * M * N + 2 * e * M * K + e * case["n"] * r * (K + N)
            f *= 3
        return {"bytes": b, "flops": f}
    b = sum(2 * (2 if t == "bf16" else 4) * n for t, n in _clip_sizes(case))
    return {"bytes": b + 4, "flops": 3 * sum(n for _, n in _clip_sizes(case))}


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = {"device": "cuda"}

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, **dev).mul_(std)

    s = {"case": dict(case)}
    if case["op"] == "ce":
        T, D, V = case["T"], case["D"], case["V"]
        w = torch.empty((V, D), dtype=torch.bfloat16, **dev)
        for part in w.split(16384):
            part.copy_(normal(part.shape[0], D, std=1.5 / math.sqrt(D)))
        labels = torch.randint(0, V, (T,), generator=g, **dev)
        # most tokens are predicted to some degree: the hidden state leans towards its label's row
        lean = torch.rand((T, 1), generator=g, **dev) * 6.0
        h = normal(T, D) + lean * w[labels].float()
        drop = torch.rand((T,), generator=g, **dev) < 0.1   # padding and prompt positions
        drop[0] = False
        labels = torch.where(drop, torch.full_like(labels, IGNORE), labels)
        s.update(h=h.bfloat16(), w=w, labels=labels, loss=torch.empty(T, **dev), lse=torch.empty(T, **dev))
        if case["grad"]:
            # the mean over the counted tokens, as a training step hands it down
            s["dloss"] = (~drop).float() / (~drop).sum()
            s["dh"] = torch.empty_like(s["h"]) if "h" in case["grad"] else None
            s["dw"] = torch.empty_like(w) if "w" in case["grad"] else None
        return s
    if case["op"] == "lora":
        M, K, N, r, n, dt = case["M"], case["K"], case["N"], case["r"], case["n"], DTYPES[case["type"]]
        if case["rows"] == "mixed":
            ids = torch.randint(0, n, (M,), generator=g, **dev)
            if n >= M:
                ids = torch.randperm(n, generator=g, **dev)[:M]
            if M > 16:   # some requests use the shared projection alone
                ids = torch.where(torch.rand((M,), generator=g, **dev) < 0.1, torch.full_like(ids, -1), ids)
        else:   # requests of ragged lengths one after another, each with its adapter
            cuts = torch.sort(torch.randint(0, M + 1, (max(0, 2 * n - 1),), generator=g, **dev)).values
            req = torch.searchsorted(cuts, torch.arange(M, **dev), right=True)
            ids = torch.randint(0, n, (2 * n,), generator=g, **dev)[req] if n > 1 else torch.zeros(M, dtype=torch.int64, **dev)
        s.update(x=normal(M, K).bfloat16(), a=normal(n, r, K, std=1 / math.sqrt(K)).bfloat16(), b=normal(n, N, r, std=1 / math.sqrt(r)).bfloat16(),
                 scale=0.5 + 1.5 * torch.rand((n,), generator=g, **dev), ids=ids.to(torch.int32), base=normal(M, N).to(dt),
                 y=torch.empty((M, N), dtype=dt, **dev), hidden=torch.empty((M, r), **dev))
        if case["train"]:
            s.update(dy=normal(M, N, std=1e-2).bfloat16(), dx_base=normal(M, K, std=1e-2).to(dt), dx=torch.empty((M, K), dtype=dt, **dev),
                     da=torch.empty((n, r, K), dtype=dt, **dev), db=torch.empty((n, N, r), dtype=dt, **dev))
        return s
    sizes = _clip_sizes(case)
    for t in ("bf16", "f32"):
        ns = [n for u, n in sizes if u == t]
        if ns:
            # tensors of one type one after another; each begins on a 16-byte boundary, as an allocator gives them
            starts, at = [], 0
            for n in ns:
                starts.append(at)
                at += (n + 7) // 8 * 8
            flat = torch.zeros(at, dtype=DTYPES[t], **dev)
            for part in flat.split(1 << 26):
                part.copy_(normal(part.numel(), std=1e-2))
            for i, n in enumerate(ns):
                flat[starts[i] + n:(starts[i + 1] if i + 1 < len(ns) else at)].zero_()
            out = torch.zeros_like(flat)
            s[t] = {"flat": flat, "out": out, "grads": [flat[b:b + n] for b, n in zip(starts, ns)], "outs": [out[b:b + n] for b, n in zip(starts, ns)]}
    s["norm"] = torch.empty(1, **dev)
    s["max_norm"] = 1.0
    return s


# ----------------------------------------------------------------------------- one pass
def _ce(s):
    import block_scaled_gemm_rfq_b200 as rfq
    case = s["case"]
    T, D, V = case["T"], case["D"], case["V"]
    g = case["grad"]
    ws = torch.empty(rfq.linear_ce_workspace_bytes(T, D, V, want_dh="h" in g, want_dw="w" in g), dtype=torch.uint8, device="cuda")
    rfq.linear_ce(s["h"], s["w"], s["labels"], s["loss"], s["lse"], ws, ignore_index=IGNORE)
    if not g:
        return {"loss": s["loss"], "lse": s["lse"]}
    rfq.linear_ce_backward(s["h"], s["w"], s["labels"], s["lse"], s["dloss"], s["dh"], s["dw"], ws, ignore_index=IGNORE)
    return {"loss": s["loss"], "lse": s["lse"], "dh": s["dh"], "dw": s["dw"]}


def _ce_plain(s):
    g = s["case"]["grad"]
    h, w, labels = s["h"].float(), s["w"].float(), s["labels"]
    logits = h @ w.T
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    kept = labels != IGNORE
    at = torch.where(kept, labels, torch.zeros_like(labels))[:, None]
    loss = torch.where(kept, (lse - logits.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    if not g:
        return {"loss": loss, "lse": lse[:, 0]}
    del logits
    d = e.div_(total)
    d.scatter_add_(1, at, torch.full_like(lse, -1.0))
    d.mul_((s["dloss"] * kept)[:, None])
    return {"loss": loss, "lse": lse[:, 0], "dh": (d @ w).bfloat16() if "h" in g else None, "dw": (d.T @ h).bfloat16() if "w" in g else None}


def _lora(s):
    import block_scaled_gemm_rfq_b200 as rfq
    case = s["case"]
    ws = torch.empty(rfq.lora_workspace_bytes(case["M"], case["K"], case["N"], case["r"], case["n"], backward=case["train"]), dtype=torch.uint8, device="cuda")
    rfq.lora(s["x"], s["a"], s["b"], s["scale"], s["ids"], s["y"], ws, base=s["base"], hidden=s["hidden"] if case["train"] else None)
    if not case["train"]:
        return {"y": s["y"]}
    rfq.lora_backward(s["x"], s["a"], s["b"], s["scale"], s["ids"], s["dy"], s["hidden"], ws, dx=s["dx"], dx_base=s["dx_base"], da=s["da"], db=s["db"])
    return {"y": s["y"], "dx": s["dx"], "da": s["da"], "db": s["db"]}


def _lora_plain(s):
    # all adapters side by side along the rank: each row keeps the columns of its own
    case = s["case"]
    N, K, r, n, dt = case["N"], case["K"], case["r"], case["n"], DTYPES[case["type"]]
    x, a, b = s["x"].float(), s["a"].float().reshape(n * r, K), s["b"].float().transpose(1, 2).reshape(n * r, N)
    of = torch.arange(n, device=x.device).repeat_interleave(r)
    keep = (s["ids"][:, None] == of[None, :]) * s["scale"].repeat_interleave(r)[None, :]
    hidden = (x @ a.T) * keep
    y = (s["base"].float() + hidden @ b).to(dt)
    if not case["train"]:
        return {"y": y}
    dy = s["dy"].float()
    dhidden = (dy @ b.T) * keep
    return {"y": y, "dx": (s["dx_base"].float() + dhidden @ a).to(dt), "da": (dhidden.T @ x).reshape(n, r, K).to(dt),
            "db": (hidden.T @ dy).reshape(n, r, N).transpose(1, 2).to(dt)}


def _clip(s):
    import block_scaled_gemm_rfq_b200 as rfq
    grads, outs = [], []
    for t in ("bf16", "f32"):
        if t in s:
            grads += s[t]["grads"]
            outs += s[t]["outs"]
    ws = torch.empty(rfq.grad_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device="cuda")
    rfq.grad_clip(grads, s["max_norm"], s["norm"], ws, outs=outs)
    return {"norm": s["norm"], **{t: s[t]["out"] for t in ("bf16", "f32") if t in s}}


def _clip_plain(s):
    # the gaps between the tensors hold zeros, so whole buffers can be taken
    flats = {t: s[t]["flat"] for t in ("bf16", "f32") if t in s}
    norm = sum(f.float().square().sum(dtype=torch.float64) for f in flats.values()).sqrt().float().reshape(1)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, **{t: (f.float() * coef).to(f.dtype) for t, f in flats.items()}}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ce": _ce, "lora": _lora, "clip": _clip}[op](state)
    return {"ce": _ce_plain, "lora": _lora_plain, "clip": _clip_plain}[op](state)


# ----------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ce":
        return _ce_exact(s, case)
    if case["op"] == "lora":
        return _lora_exact(s, case)
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in ("bf16", "f32"):
        for v in s[t]["grads"] if t in s else []:
            total += torch.linalg.vector_norm(v.double()) ** 2
    norm = total.sqrt()
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return {"norm": norm.reshape(1), **{t: s[t]["flat"].double() * coef for t in ("bf16", "f32") if t in s}}


def _ce_exact(s, case):
    T, D, V, g = case["T"], case["D"], case["V"], case["grad"]
    w, labels = s["w"].double(), s["labels"]
    loss, lse, dh, dw = [], [], [], (torch.zeros((V, D), dtype=torch.float64, device="cuda") if "w" in g else None)
    for b in range(0, T, 512):   # token by token the definition is the same: rows in groups, for memory
        h, lab = s["h"][b:b + 512].double(), labels[b:b + 512]
        z = torch.mm(h, w.t())
        part = torch.logsumexp(z, dim=1)
        counted = lab.ne(IGNORE)
        rows = torch.nonzero(counted)[:, 0]
        one = torch.zeros_like(part)
        one[rows] = part[rows] - z[rows, lab[rows]]
        loss.append(one)
        lse.append(part)
        if g:
            p = torch.exp(z - part[:, None])
            p[rows, lab[rows]] -= 1.0
            p *= (s["dloss"][b:b + 512].double() * counted)[:, None]
            if "h" in g:
                dh.append(torch.mm(p, w))
            if "w" in g:
                dw.addmm_(p.t(), h)
    if not g:
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    return {"loss": torch.cat(loss), "lse": torch.cat(lse), "dh": torch.cat(dh) if dh else None, "dw": dw}


def _lora_exact(s, case):
    n, r = case["n"], case["r"]
    y = s["base"].double()
    dx = s["dx_base"].double() if case["train"] else None
    da, db = [], []
    for k in range(n):   # one adapter after another, on its rows alone
        rows = torch.nonzero(s["ids"] == k)[:, 0]
        a, b, c = s["a"][k].double(), s["b"][k].double(), float(s["scale"][k])
        x = s["x"][rows].double()
        u = torch.mm(x, a.t())
        y[rows] += c * torch.mm(u, b.t())
        if case["train"]:
            dy = s["dy"][rows].double()
            v = c * torch.mm(dy, b)
            dx[rows] += torch.mm(v, a)
            da.append(torch.mm(v.t(), x))
            db.append(c * torch.mm(dy.t(), u))
    if not case["train"]:
        return {"y": y}
    return {"y": y, "dx": dx, "da": torch.stack(da), "db": torch.stack(db)}
