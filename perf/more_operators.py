"""The operators of a mixture-of-experts block's training pass, as cases to be measured: the gradients of combine and
dispatch, the experts' products in bf16 with theirs, and the norm and clipping of all gradients.

Each case is one call, or the two that belong together, at a size of this library's workloads or of the range around
them. With ``own`` false ``run`` computes it by elementary torch operations, with ``own`` true by the library.
"""

import math

import numpy as np
import torch

own = False


def listed():
    return [
        # a small batch, per expert: latency
        dict(name="combine backward small", op="combine_back", ll=True, T=128, H=7168, E=256, R=32, k=8, padded=False),
        # a training batch, per rank: its rows' and its gates' gradients
        dict(name="combine backward train", op="combine_back", ll=False, T=4096, H=7168, E=256, R=32, k=8, padded=True),
        # a training batch, per rank, with the gradient that reaches the tokens by the router
        dict(name="dispatch backward train", op="dispatch_back", ll=False, T=4096, H=7168, E=256, R=32, k=8, padded=True,
             other=True, gates=False),
        # odd sizes, per expert, gates that went with the rows
        dict(name="dispatch backward ragged", op="dispatch_back", ll=True, T=1531, H=2184, E=48, R=8, k=6, padded=True,
             other=False, gates=True),
        # one row at each expert: a weight stream
        dict(name="product one row", op="product", G=8, M=8, K=1792, N=7168, spread="one"),
        # a training batch's rows at one GPU's experts, unequal counts
        dict(name="product train", op="product", G=8, M=8192, K=1792, N=7168, spread="skewed"),
        # its gradients, the weights' in bf16
        dict(name="product backward train", op="product_back", G=8, M=8192, K=1792, N=7168, spread="skewed", half=True),
        # odd sizes: short experts, products that end inside every tile
        dict(name="gate up ragged", op="gate_up", G=24, M=1531, K=2184, N=1808, spread="skewed", keep=True),
        # the first product's gradients on a training batch, the weights' in float
        dict(name="gate up backward train", op="gate_up_back", G=8, M=8192, K=7168, N=3584, spread="skewed", half=False),
        # a small model's gradients: a few dozen tensors, latency
        dict(name="clip small", op="clip", count=24, total=200000, half=0.5, into=True, clipped=True),
        # a thousand tensors of every size, in both types: the norm alone, to be summed over the GPUs before the clip
        dict(name="norm of many", op="clip", count=1000, total=60000000, half=0.7, into=False, clipped=False),
        # one layer's experts and what is around them: the clipped gradients go to the optimiser's own buffers
        dict(name="clip experts", op="clip", count=40, total=308000000, half=0.99, into=True, clipped=True),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["combine_back", "dispatch_back", "product", "product_back", "gate_up", "gate_up_back", "clip"])
    if op in ("combine_back", "dispatch_back"):
        H, R = 8 * _span(rng, 4, 1024), 1 << rng.randint(0, 6)
        E = R * _span(rng, 1, 256 // R)
        k = rng.randint(1, min(E, 16))
        c = dict(op=op, ll=rng.random() < 0.5, T=_span(rng, 1, min(16384, 4096 * 8 * 7168 // (k * H))), H=H, E=E, R=R,
                 k=k, padded=rng.random() < 0.5)
        if op == "dispatch_back":
            c.update(other=rng.random() < 0.5, gates=rng.random() < 0.5)
        return c
    if op == "clip":
        count = _span(rng, 1, 1000)
        total, into = max(count, _span(rng, 1, 300000000)), rng.random() < 0.6
        half = rng.choice([0.0, 0.5, 0.9, 1.0])
        return dict(op=op, count=count, total=int(total * (0.5 + 0.5 * half)), half=half, into=into,
                    clipped=into and rng.random() < 0.7)
    G, M = _span(rng, 1, 32), _span(rng, 1, 8192)
    N = 8 * _span(rng, 8, 448) if op.startswith("product") else 16 * _span(rng, 4, 224)
    K = 8 * _span(rng, 8, min(896, 8 * 896 * 3584 // (G * N)))
    c = dict(op=op, G=G, M=M, K=K, N=N, spread="one" if M == G else rng.choice(["even", "skewed", "skewed"]))
    if op == "gate_up":
        c["keep"] = rng.random() < 0.7
    elif op.endswith("back"):
        c["half"] = rng.random() < 0.5
    return c


def work(case):
    c = case
    if c["op"] in ("combine_back", "dispatch_back"):
        T, H, k = c["T"], c["H"], c["k"]
        # a token's rows: its choices, or the ranks that k different experts meet, on average
        per = c["E"] // c["R"]
        rows = T * (k if c["ll"] else c["R"] * (1 - math.comb(c["E"] - per, k) / math.comb(c["E"], k)))
        rows *= 0.95 if c["padded"] else 1.0
        if c["op"] == "combine_back":
            return {"bytes": int(rows * 4 * H + T * 2 * H + T * k * 12), "flops": int(3 * rows * H)}
        return {"bytes": int(rows * 2 * H + T * H * (4 if c["other"] else 2) + T * k * (12 if c["gates"] else 4)),
                "flops": int(rows * H)}
    if c["op"] == "clip":
        item = 4 - 2 * c["half"]
        return {"bytes": int(c["total"] * item * (2 if c["into"] else 1)), "flops": int(c["total"] * (3 if c["into"] else 2))}
    K, N, M = c["K"], c["N"], c["M"]
    kept = M if c["spread"] == "one" else M - M // 16
    weights = min(c["G"], max(kept, 1)) * K * N
    if c["op"] == "product":
        return {"bytes": 2 * weights + 2 * kept * (K + N), "flops": 2 * kept * K * N}
    if c["op"] == "gate_up":
        return {"bytes": 2 * weights + kept * (2 * K + N + (2 * N if c["keep"] else 0)), "flops": 2 * kept * K * N}
    grad_w = c["G"] * K * N * (2 if c["half"] else 4)
    if c["op"] == "product_back":
        return {"bytes": 2 * weights + grad_w + kept * (4 * K + 2 * N), "flops": 4 * kept * K * N}
    return {"bytes": 2 * weights + grad_w + kept * (4 * K + 2 * N + N + 2 * N), "flops": 4 * kept * K * N}


# ---- inputs -----------------------------------------------------------------------------------------------------


def _counts(case, seed):
    """Rows of each expert: one each, about equal, or falling off as 1 / rank with the order shuffled."""
    G, M = case["G"], case["M"]
    if case["spread"] == "one":
        return np.ones(G, np.int64)
    r = np.random.RandomState(seed % (1 << 31))
    p = np.ones(G) if case["spread"] == "even" else r.permutation(1.0 / np.arange(1, G + 1))
    return r.multinomial(M - M // 16, p / p.sum())


def _layout(c, idx):
    """Rows of a dispatch: [T, k] per expert (the choices in the order of their experts), [T, R] per rank (each rank's
    tokens in their order); -1 where there is none."""
    T, E, R = c["T"], c["E"], c["R"]
    if c["ll"]:
        flat = idx.view(-1)
        order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
        slot = torch.empty_like(order)
        slot[order] = torch.arange(order.numel(), device="cuda")
        return torch.where(flat < 0, -1, slot).view(T, -1).int()
    there = torch.zeros(T, R + 1, dtype=torch.int64, device="cuda")
    there.scatter_(1, torch.where(idx < 0, R, idx.long() // (E // R)), 1)
    there = there[:, :R].t().reshape(-1)
    slot = torch.where(there != 0, there.cumsum(0) - 1, -1).view(R, T).t().contiguous()
    return slot.int()


def _sizes(c):
    """Sizes of a clip's tensors, those of one model: spread over three factors of ten, `total` together; and which are
    bf16."""
    n, total = c["count"], c["total"]
    r = np.random.RandomState((n * 1000003 + total) % (1 << 31))
    p = np.exp(r.uniform(0.0, math.log(1000.0), n))
    size = 1 + np.floor((total - n) * p / p.sum()).astype(np.int64)
    order = np.argsort(-size)
    half, got = np.zeros(n, bool), 0     # the largest first, while they stay within their share
    for i in order:
        if got + size[i] <= c["half"] * total * (1 + 1e-9):
            half[i], got = True, got + size[i]
    return size, half


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    bf = dict(dtype=torch.bfloat16, device="cuda")
    s = {"case": c}
    if c["op"] in ("combine_back", "dispatch_back"):
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        logits = 1.5 * randn(T, E) + 0.5 * randn(E)
        v, idx = torch.topk(logits, k, dim=1)
        if c["padded"]:    # padded tokens and dropped choices
            idx = torch.where((rand(T, 1) < 0.04) | (rand(T, k) < 0.01), -1, idx)
        s["idx"] = idx.int().contiguous()
        s["w"] = torch.where(idx < 0, 0.0, torch.softmax(v, 1)).contiguous()
        s["slot"] = _layout(c, s["idx"])
        s["rows"] = rows = T * (k if c["ll"] else min(k, c["R"]))    # that the buffers hold; the last ones may be no token's
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if c["op"] == "combine_back":
            s["y"] = randn(rows, H).bfloat16()
            s["grad_out"] = (0.1 * randn(T, H)).bfloat16()
            s["grad_y"] = torch.zeros(rows, H, **bf)
            s["grad_w"] = torch.empty(T, k, device="cuda")
        else:
            s["grad_rows"] = (0.1 * randn(rows, H)).bfloat16()
            s["other"] = (0.1 * randn(T, H)).bfloat16() if c["other"] else None
            s["grad_gates"] = None
            if c["gates"]:    # of the gates that went with the rows: one a row, or a rank's of the token's choices
                s["grad_gates"] = randn(rows) if c["ll"] else randn(rows, k)
            s["grad_x"] = torch.empty(T, H, **bf)
            s["grad_w"] = torch.empty(T, k, device="cuda") if c["gates"] else None
        if own:
            import combine_topk_rank_amd as ep
            s["shape"] = ep.shape(T, H, E, c["R"], k)
        return s
    if c["op"] == "clip":
        size, half = _sizes(c)
        # the gradients of a type lie in one buffer, each from a multiple of 16 bytes on, but every fifth right behind
        # the one before it
        at, end = np.zeros(c["count"], np.int64), {True: 0, False: 0}
        for i in range(c["count"]):
            step = 1 if i % 5 == 4 else 8 if half[i] else 4
            at[i] = -(-end[half[i]] // step) * step
            end[half[i]] = at[i] + size[i]
        for key, kind in ((True, torch.bfloat16), (False, torch.float32)):
            flat = torch.zeros(int(end[key]), dtype=kind, device="cuda")
            for i in np.flatnonzero(half == key):
                flat[at[i]:at[i] + size[i]].copy_(randn(int(size[i])) * float(10.0 ** (-2 - i % 3)))
            s["half" if key else "full"] = flat
            s["half_into" if key else "full_into"] = torch.zeros_like(flat) if c["into"] else None
        where = [("half" if half[i] else "full", int(at[i]), int(at[i] + size[i])) for i in range(c["count"])]
        norm = math.sqrt(sum(float(s[n].double().square().sum()) for n in ("half", "full")))
        s["bound"] = 0.3 * norm if c["clipped"] else 2.0 * norm + 1.0
        s["sum_squares"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        s["norm"] = torch.zeros(1, device="cuda")
        if own:
            import combine_topk_rank_amd as ep
            s["tensors"] = ep.TensorList([s[n][a:b] for n, a, b in where])
            s["into"] = ep.TensorList([s[n + "_into"][a:b] for n, a, b in where]) if c["into"] else None
            s["workspace"] = torch.zeros(max(16, ep.ep_grad_norm_workspace_bytes(s["tensors"])), dtype=torch.uint8, device="cuda")
        return s
    G, M, K, N = c["G"], c["M"], c["K"], c["N"]
    counts = _counts(c, seed)
    s["most"] = int(max(counts.max(), M - counts.sum(), 1))
    s["offset"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    s["rows"] = (randn(M, K) * (0.5 + rand(M, 1))).bfloat16()
    s["w"] = torch.empty(G, N, K, **bf)
    for g in range(G):
        s["w"][g] = (randn(N, K) * K ** -0.5).bfloat16()
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if c["op"] == "product":
        s["out"] = torch.zeros(M, N, **bf)
    elif c["op"] == "gate_up":
        s["pre"] = torch.zeros(M, N, **bf) if c["keep"] else None
        s["out"] = torch.zeros(M, N // 2, **bf)
    else:
        s["grad_out"] = (0.1 * randn(M, N if c["op"] == "product_back" else N // 2)).bfloat16()
        s["grad_rows"] = torch.zeros(M, K, **bf)
        s["grad_w"] = torch.empty(G, N, K, dtype=torch.bfloat16 if c["half"] else torch.float32, device="cuda")
        if c["op"] == "gate_up_back":    # what the forward call left
            s["pre"] = _grouped(s, s["rows"].float(), s["w"].float().transpose(1, 2).contiguous()).bfloat16()
            s["grad_pre"] = torch.zeros(M, N, **bf)
        if own:
            import combine_topk_rank_amd as ep
            s["workspace"] = torch.zeros(max(16, ep.ep_expert_backward_workspace_bytes(G, M, N, K)), dtype=torch.uint8,
                                         device="cuda")
    return s


# ---- the operators in elementary operations ---------------------------------------------------------------------


def _choices(s):
    """Each choice's row [T, k] (0 without one), which have one, and, per rank, which are their rank's first of the token."""
    c = s["case"]
    kept = s["idx"] >= 0
    if c["ll"]:
        return s["slot"].clamp_min(0).long(), kept, kept, None
    rank = torch.where(kept, s["idx"].long() // (c["E"] // c["R"]), -1)
    same = rank[:, :, None] == rank[:, None, :]
    earlier = torch.ones(c["k"], c["k"], dtype=torch.bool, device="cuda").tril(-1)
    return s["slot"].gather(1, rank.clamp_min(0)).clamp_min(0).long(), kept, kept & ~(same & earlier).any(2), same


def _combine_back(s):
    row, kept, first, same = _choices(s)
    T, k = row.shape
    H, rows = s["case"]["H"], s["rows"]
    g = s["grad_out"].float()
    w = torch.where(kept, s["w"], 0.0)
    if same is not None:     # a rank's weight: that of all the token's choices there
        w = (same.float() * w[:, None, :]).sum(2)
    grad_y = torch.zeros(rows + 1, H, device="cuda")      # one more, for choices without a row
    grad_y[torch.where(first, row, rows).view(-1)] = (w[:, :, None] * g[:, None, :]).view(T * k, H)
    dots = (torch.cat([s["y"], s["y"].new_zeros(1, H)])[row].float() * g[:, None, :]).sum(2)
    return {"grad_y": grad_y[:rows].bfloat16(), "grad_w": torch.where(kept, dots, 0.0)}


def _dispatch_back(s):
    row, kept, first, _ = _choices(s)
    H = s["case"]["H"]
    v = torch.cat([s["grad_rows"], s["grad_rows"].new_zeros(1, H)])[torch.where(first, row, s["rows"])].float().sum(1)
    if s["other"] is not None:
        v = v + s["other"].float()
    out = {"grad_x": v.bfloat16()}
    if s["grad_gates"] is not None:
        gates = torch.cat([s["grad_gates"], s["grad_gates"].new_zeros(1, *s["grad_gates"].shape[1:])])
        gates = gates[row]
        if gates.dim() == 3:
            gates = gates.diagonal(dim1=1, dim2=2)
        out["grad_w"] = torch.where(kept, gates, 0.0)
    return out


def _place(s):
    """Each row's expert (G: none) and its number among that expert's rows."""
    row = torch.arange(s["case"]["M"], device="cuda", dtype=torch.int32)
    g = torch.searchsorted(s["offset"], row, right=True) - 1
    return g, (row - s["offset"][g]).long()


def _spread_out(s, x):
    """Rows by expert, [G, most, width], zeros behind an expert's last."""
    G = s["case"]["G"]
    g, at = _place(s)
    a = torch.zeros(G + 1, s["most"], x.shape[1], device="cuda")
    a[g, at] = x
    return a[:G]


def _grouped(s, x, b):
    """Each row of x times its expert's [K, N], in float; rows without an expert: zero."""
    g, at = _place(s)
    y = torch.bmm(_spread_out(s, x), b)[g.clamp_max(s["case"]["G"] - 1), at]
    return torch.where((g < s["case"]["G"])[:, None], y, 0.0)


def _forward(s):
    y = _grouped(s, s["rows"].float(), s["w"].float().transpose(1, 2).contiguous())
    if s["case"]["op"] == "product":
        return {"out": y.bfloat16()}
    gate, up = y[:, :s["case"]["N"] // 2], y[:, s["case"]["N"] // 2:]
    out = {"out": (gate / (1.0 + torch.exp(-gate)) * up).bfloat16()}
    if s["pre"] is not None:
        out["pre"] = y.bfloat16()
    return out


def _backward(s):
    c, d, out = s["case"], s["grad_out"].float(), {}
    if c["op"] == "gate_up_back":
        gate, up = s["pre"][:, :c["N"] // 2].float(), s["pre"][:, c["N"] // 2:].float()
        sg = 1.0 / (1.0 + torch.exp(-gate))
        d = torch.cat([d * up * sg * (1.0 + gate * (1.0 - sg)), d * gate * sg], 1).bfloat16()
        g, _ = _place(s)
        d = torch.where((g < c["G"])[:, None], d, 0.0)
        out["grad_pre"] = d
        d = d.float()
    out["grad_rows"] = _grouped(s, d, s["w"].float()).bfloat16()
    grad_w = torch.bmm(_spread_out(s, d).transpose(1, 2).contiguous(), _spread_out(s, s["rows"].float()))
    out["grad_w"] = grad_w.to(s["grad_w"].dtype)
    return out


def _clip(s):
    # squares of a float and their sums in 64 bits, or a large or small gradient would be lost
    total = s["half"].double().square().sum() + s["full"].double().square().sum()
    norm = total.sqrt()
    out = {"sum_squares": total.view(1), "norm": norm.float().view(1)}
    if s["case"]["into"]:
        scale = torch.where(norm > s["bound"], s["bound"] / norm, 1.0).float()
        out["half"] = (s["half"].float() * scale).bfloat16()
        out["full"] = s["full"] * scale
    return out


# ---- the operators by the library -------------------------------------------------------------------------------


def _own(s):
    import combine_topk_rank_amd as ep
    c = s["case"]
    op = c["op"]
    if op == "combine_back":
        call = ep.ep_combine_ll_backward if c["ll"] else ep.ep_combine_backward
        call(s["shape"], s["y"], s["idx"], s["w"], s["slot"], s["grad_out"], s["grad_y"], s["grad_w"], s["status"])
        return {"grad_y": s["grad_y"], "grad_w": s["grad_w"]}
    if op == "dispatch_back":
        call = ep.ep_dispatch_ll_backward if c["ll"] else ep.ep_dispatch_backward
        call(s["shape"], s["idx"], s["slot"], s["grad_rows"], s["grad_gates"], s["other"], s["grad_x"], s["grad_w"],
             s["status"])
        return {"grad_x": s["grad_x"], **({"grad_w": s["grad_w"]} if c["gates"] else {})}
    if op == "product":
        ep.ep_expert_product_bf16(s["rows"], s["offset"], s["w"], s["out"], s["status"])
        return {"out": s["out"]}
    if op == "gate_up":
        ep.ep_expert_gate_up_bf16(s["rows"], s["offset"], s["w"], s["pre"], s["out"], s["status"])
        return {"out": s["out"], **({"pre": s["pre"]} if c["keep"] else {})}
    if op == "product_back":
        ep.ep_expert_product_bf16_backward(s["rows"], s["offset"], s["w"], s["grad_out"], s["grad_rows"], s["grad_w"],
                                           s["status"], s["workspace"])
        return {"grad_rows": s["grad_rows"], "grad_w": s["grad_w"]}
    if op == "gate_up_back":
        ep.ep_expert_gate_up_bf16_backward(s["rows"], s["offset"], s["w"], s["pre"], s["grad_out"], s["grad_pre"],
                                           s["grad_rows"], s["grad_w"], s["status"], s["workspace"])
        return {"grad_pre": s["grad_pre"], "grad_rows": s["grad_rows"], "grad_w": s["grad_w"]}
    ep.ep_grad_norm(s["tensors"], s["sum_squares"], s["norm"], s["workspace"])
    out = {"sum_squares": s["sum_squares"], "norm": s["norm"]}
    if c["into"]:
        ep.ep_grad_clip(s["tensors"], s["sum_squares"], s["bound"], s["into"])
        out.update(half=s["half_into"], full=s["full_into"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"combine_back": _combine_back, "dispatch_back": _dispatch_back, "product": _forward, "gate_up": _forward,
            "product_back": _backward, "gate_up_back": _backward, "clip": _clip}[state["case"]["op"]](state)


# ---- the operators in 64 bits -----------------------------------------------------------------------------------


def _exact_exchange(s):
    """Gradients by differentiating dispatch and combine themselves, a rank (or a choice) after the other."""
    c = s["case"]
    T, H, k = c["T"], c["H"], c["k"]
    token = torch.arange(T, device="cuda")
    parts = []     # tokens, their rows, and which of their choices these rows serve
    for i in range(k if c["ll"] else c["R"]):
        if c["ll"]:
            serves = torch.zeros(T, k, dtype=torch.bool, device="cuda")
            serves[:, i] = s["idx"][:, i] >= 0
        else:
            serves = (s["idx"] >= 0) & (torch.div(s["idx"], c["E"] // c["R"], rounding_mode="floor") == i)
        there = serves.any(1)
        parts.append((token[there], s["slot"][there, i].long(), serves[there].double()))
    if c["op"] == "combine_back":
        w = s["w"].double().requires_grad_(True)
        grad_y = torch.zeros(s["rows"], H, dtype=torch.float64, device="cuda")
        grad_w = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for t, row, serves in parts:
            y = s["y"][row].double().requires_grad_(True)
            out = (w[t] * serves).sum(1, keepdim=True) * y
            dy, dw = torch.autograd.grad(out, (y, w), s["grad_out"][t].double())
            grad_y[row] = dy
            grad_w += dw
        return {"grad_y": grad_y, "grad_w": grad_w}
    x = torch.zeros(T, H, dtype=torch.float64, device="cuda") if s["other"] is None else s["other"].double()
    out = {"grad_x": x}
    if s["grad_gates"] is not None:
        out["grad_w"] = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for t, row, serves in parts:
        x.index_add_(0, t, s["grad_rows"][row].double())
        if s["grad_gates"] is not None:
            gates = s["grad_gates"][row].double()
            out["grad_w"][t] += serves * (gates[:, None] if c["ll"] else gates)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("combine_back", "dispatch_back"):
        return _exact_exchange(s)
    if c["op"] == "clip":
        norms = [torch.linalg.vector_norm(s[n].double()) if s[n].numel() else torch.zeros((), dtype=torch.float64, device="cuda")
                 for n in ("half", "full")]
        norm = torch.hypot(*norms)
        out = {"sum_squares": (norms[0] ** 2 + norms[1] ** 2).view(1), "norm": norm.view(1)}
        if c["into"]:
            part = min(1.0, s["bound"] / float(norm)) if float(norm) else 1.0
            out.update(half=s["half"].double() * part, full=s["full"].double() * part)
        return out
    back, M, K, N = c["op"].endswith("back"), c["M"], c["K"], c["N"]
    wide = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")  # noqa: E731
    gate = c["op"].startswith("gate")
    if back:
        # in float, the gradient of weights whose product's own was rounded on the way hangs on that rounding's ties
        out = {"grad_rows": wide(M, K), "grad_w": None if gate and not c["half"] else wide(c["G"], N, K)}
        if gate:
            out["grad_pre"] = wide(M, N)
    else:
        out = {"out": wide(M, N // 2 if gate else N)}
        if gate and c["keep"]:
            out["pre"] = wide(M, N)
    bounds = s["offset"].tolist()
    for g in range(c["G"]):
        at = slice(bounds[g], bounds[g + 1])
        if at.start == at.stop:
            continue
        x, w = s["rows"][at].double(), s["w"][g].double()
        if back:
            d = s["grad_out"][at].double()
            if gate:     # the products' gradients are those of the rounded one
                pre = s["pre"][at].double().requires_grad_(True)
                y = torch.nn.functional.silu(pre[:, :N // 2]) * pre[:, N // 2:]
                d, = torch.autograd.grad(y, pre, d)
                out["grad_pre"][at] = d
                d = d.bfloat16().double()
            out["grad_rows"][at] = d @ w
            if out["grad_w"] is not None:
                out["grad_w"][g] = d.t().contiguous() @ x
            continue
        y = x @ w.t().contiguous()
        if "pre" in out:
            out["pre"][at] = y
        out["out"][at] = torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:] if gate else y
    return out
