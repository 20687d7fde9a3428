"""The operators around a dispatch and a combine, as cases to be measured: the norm that makes the rows, the router that
names their experts, and the two expert products between dispatch and combine.

Each case is one call (forward or backward) at a size of this library's workloads or of the range around them. With
``own`` false ``run`` computes it by elementary torch operations, with ``own`` true by the library.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128          # elements that share a scale, in rows; weights share one per 128 x 128
FP8_MAX = 448.0      # largest e4m3 value
AMAX_MIN = 1e-4      # least block maximum of a quantised row
EPS = 1e-6           # of the norm
SOFTMAX, RENORM = 0, 1


def listed():
    return [
        # one token of a decoding step, between two layers
        dict(name="norm one token", op="norm", T=1, H=7168, residual=True, rows=True, y=True, rstd=False),
        # a decoding batch
        dict(name="norm decode", op="norm", T=128, H=7168, residual=True, rows=True, y=True, rstd=False),
        # a long prompt or a training batch: the residual stream, the router's input and the 8-bit rows in one call
        dict(name="norm prompt", op="norm", T=16384, H=7168, residual=True, rows=True, y=True, rstd=True),
        # the training batch's backward, with the residual stream's own gradient
        dict(name="norm backward", op="norm_back", T=4096, H=7168, residual=True),
        # a decoding batch's choice of experts: no balance loss
        dict(name="route decode", op="route", T=128, E=256, k=8, mode=RENORM, half=True, balance=False, masked=False),
        # a training batch with padded tokens: choices, counts and balance loss
        dict(name="route train", op="route", T=16384, E=256, k=8, mode=RENORM, half=False, balance=True, masked=True),
        # its backward: the gates' gradient and the balance loss's
        dict(name="route backward", op="route_back", T=16384, E=256, k=8, mode=RENORM, half=False, balance=True, masked=True),
        # one token's eight experts, all of them here: one product, a weight stream
        dict(name="product one token", op="product", G=8, M=8, K=1792, N=7168, spread="one"),
        # a training batch's rows at one GPU's experts, unequal counts
        dict(name="product train", op="product", G=8, M=8192, K=1792, N=7168, spread="skewed"),
        # a decoding batch over many experts, some without a row: both products and the gate between them
        dict(name="experts decode", op="experts", G=32, M=128, H=7168, F=1792, spread="skewed"),
        # odd sizes: short experts, products that end inside every tile
        dict(name="experts ragged", op="experts", G=24, M=1531, H=2176, F=896, spread="skewed"),
        # a training batch's rows at one GPU's experts
        dict(name="experts train", op="experts", G=8, M=8192, H=7168, F=1792, spread="skewed"),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "route", "route_back", "product", "experts", "product", "experts"])
    if op in ("norm", "norm_back"):
        rows = op == "norm" and rng.random() < 0.6
        H = 128 * _span(rng, 1, 64) if rows else 8 * _span(rng, 8, 1024)
        c = dict(op=op, T=_span(rng, 1, min(16384, 117440512 // H // (1 if op == "norm" else 2))), H=H,
                 residual=rng.random() < 0.7)
        if op == "norm":
            y = not rows or rng.random() < 0.7
            c.update(rows=rows, y=y, rstd=rng.random() < 0.5)
        return c
    if op in ("route", "route_back"):
        E = rng.choice([_span(rng, 4, 512), 64, 256])
        return dict(op=op, T=_span(rng, 1, min(16384, 4194304 // E)), E=E, k=rng.randint(1, min(E, 16)),
                    mode=rng.choice([SOFTMAX, RENORM]), half=rng.random() < 0.5,
                    balance=op == "route_back" or rng.random() < 0.6, masked=rng.random() < 0.5)
    G, M = _span(rng, 1, 32), _span(rng, 1, 8192)
    spread = "one" if M == G else rng.choice(["even", "skewed", "skewed"])
    if op == "product":   # any width of whole 16-byte rows
        return dict(op=op, G=G, M=M, K=128 * _span(rng, 1, 56), N=8 * _span(rng, 8, 896), spread=spread)
    return dict(op=op, G=G, M=M, H=128 * _span(rng, 1, 56), F=128 * _span(rng, 1, 14), spread=spread)


def work(case):
    c = case
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        per = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0) + (1 + 4 / BLOCK if c["rows"] else 0)
        return {"bytes": T * H * per + 4 * H + (4 * T if c["rstd"] else 0), "flops": 8 * T * H}
    if c["op"] == "norm_back":
        T, H = c["T"], c["H"]
        return {"bytes": T * H * (6 + (2 if c["residual"] else 0)) + 8 * H + 4 * T, "flops": 10 * T * H}
    if c["op"] in ("route", "route_back"):
        T, E, k = c["T"], c["E"], c["k"]
        item = 2 if c["half"] else 4
        if c["op"] == "route":
            return {"bytes": T * E * item + T * k * 8 + (T * 4 + E * 4 if c["balance"] else 0), "flops": 4 * T * E}
        return {"bytes": 2 * T * E * item + T * k * 12 + T * 4 + E * 4, "flops": 6 * T * E}
    kept = c["M"] if c["spread"] == "one" else c["M"] - c["M"] // 16
    K, N = (c["K"], c["N"]) if c["op"] == "product" else (c["H"], c["H"])
    weights = K * N if c["op"] == "product" else 3 * c["H"] * c["F"]
    return {"bytes": min(c["G"], kept) * weights * (1 + 4 / BLOCK / BLOCK) + kept * (K * (1 + 4 / BLOCK) + 2 * N),
            "flops": 2 * kept * weights}


# ---- inputs -----------------------------------------------------------------------------------------------------


def _row_bytes(H):
    """Bytes of one 8-bit row: H codes, a float scale per 128 of them, zero bytes up to a multiple of 128."""
    return -(-(H + 4 * (H // BLOCK)) // 128) * 128


def _rows8(v):
    """[M, H] floats as 8-bit rows, the form that the dispatch sends."""
    M, H = v.shape
    b = v.float().view(M, H // BLOCK, BLOCK)
    a = b.abs().amax(2).clamp_min(AMAX_MIN)
    rows = torch.zeros(M, _row_bytes(H), dtype=torch.uint8, device=v.device)
    rows[:, :H] = (b * (FP8_MAX / a)[:, :, None]).view(M, H).to(torch.float8_e4m3fn).view(torch.uint8)
    rows[:, H:H + H // 32] = (a / FP8_MAX).view(torch.uint8)
    return rows


def _weights8(G, N, K, gen):
    """Expert weights in 8 bits with a scale per 128 x 128 block: codes [G, N, K], scales [G, ceil(N / 128), K / 128]."""
    nb = -(-N // BLOCK)
    codes = torch.empty(G, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(G, nb, K // BLOCK, dtype=torch.float32, device="cuda")
    for g in range(G):
        w = torch.zeros(nb * BLOCK, K, device="cuda")
        w[:N].normal_(0.0, K ** -0.5, generator=gen)
        w = w.view(nb, BLOCK, K // BLOCK, BLOCK)
        s = w.abs().amax((1, 3)) / FP8_MAX
        codes[g] = (w / s[:, None, :, None]).reshape(nb * BLOCK, K)[:N].to(torch.float8_e4m3fn)
        scales[g] = s
    return codes, scales


def _counts(case, seed):
    """Rows of each expert: one each, about equal, or falling off as 1 / rank with the order shuffled."""
    G, M = case["G"], case["M"]
    if case["spread"] == "one":
        return np.ones(G, np.int64)
    r = np.random.RandomState(seed % (1 << 31))
    p = np.ones(G) if case["spread"] == "even" else r.permutation(1.0 / np.arange(1, G + 1))
    return r.multinomial(M - M // 16, p / p.sum())


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": c}
    if c["op"] in ("norm", "norm_back"):
        T, H = c["T"], c["H"]
        stream = 1.0 + 4.0 * (rand(H) < 0.01)   # a few channels of the residual stream are large
        s["x"] = (randn(T, H) * stream).bfloat16()
        s["weight"] = 1.0 + 0.1 * randn(H)
        if c["op"] == "norm":
            s["residual"] = (2.0 * randn(T, H) * stream).bfloat16() if c["residual"] else None
            s["residual_out"] = torch.empty_like(s["x"]) if c["residual"] else None
            s["y"] = torch.empty_like(s["x"]) if c["y"] else None
            s["rows"] = torch.zeros(T, _row_bytes(H), dtype=torch.uint8, device="cuda") if c["rows"] else None
            s["rstd"] = torch.empty(T, device="cuda") if c["rstd"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
            s["grad_y"] = (0.1 * randn(T, H)).bfloat16()
            s["grad_residual"] = (0.1 * randn(T, H)).bfloat16() if c["residual"] else None
            s["grad_x"] = torch.empty_like(s["x"])
            s["grad_weight"] = torch.empty(H, device="cuda")
            if own:
                import combine_topk_rank_amd as ep
                s["workspace"] = torch.zeros(max(16, ep.ep_rmsnorm_workspace_bytes(T, H)), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] in ("route", "route_back"):
        T, E, k = c["T"], c["E"], c["k"]
        kind = torch.bfloat16 if c["half"] else torch.float32
        s["mask"] = (rand(T) < 0.95).to(torch.uint8) if c["masked"] else None
        logits = 1.5 * randn(T, E) + 0.5 * randn(E)
        if c["masked"]:   # a padded token's logits are whatever its memory held
            logits = torch.where((s["mask"] != 0)[:, None], logits, math.nan)
        s["logits"] = logits.to(kind)
        s["idx"] = torch.empty(T, k, **i32)
        s["w"] = torch.empty(T, k, device="cuda")
        b = c["balance"]
        s["counts"] = torch.empty(E, **i32) if b else None
        s["kept"] = torch.empty(1, **i32) if b else None
        s["lse"] = torch.empty(T, device="cuda") if b else None
        s["loss"] = torch.empty(1, device="cuda") if b else None
        if own:
            import combine_topk_rank_amd as ep
            s["workspace"] = torch.zeros(max(16, ep.ep_route_workspace_bytes(T, E)), dtype=torch.uint8, device="cuda")
        if c["op"] == "route_back":   # what the forward call left
            f = _route(s)
            s.update(idx=f["idx"], w=f["w"], counts=f["counts"], kept=f["kept"], lse=f["lse"])
            s["grad_w"] = randn(T, k)
            s["grad_loss"] = torch.full((1,), 0.01, device="cuda")
            s["grad_logits"] = torch.empty_like(s["logits"])
        return s
    G, M = c["G"], c["M"]
    counts = _counts(c, seed)
    s["most"] = int(max(counts.max(), M - counts.sum(), 1))
    s["offset"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), **i32)
    K = c["K"] if c["op"] == "product" else c["H"]
    s["rows"] = _rows8((randn(M, K) * (0.5 + rand(M, 1))).bfloat16())
    if c["op"] == "product":
        s["codes"], s["scales"] = _weights8(G, c["N"], K, gen)
        s["out"] = torch.zeros(M, c["N"], dtype=torch.bfloat16, device="cuda")
    else:
        s["codes"], s["scales"] = _weights8(G, 2 * c["F"], K, gen)      # an expert's gate, then its up
        s["codes2"], s["scales2"] = _weights8(G, K, c["F"], gen)
        s["inner"] = torch.zeros(M, _row_bytes(c["F"]), dtype=torch.uint8, device="cuda")
        s["out"] = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    s["status"] = torch.zeros(1, **i32)
    return s


# ---- the operators in elementary operations ---------------------------------------------------------------------


def _quantise(v):
    """Codes and scales of [M, H] floats."""
    M, H = v.shape
    b = v.view(M, H // BLOCK, BLOCK)
    a = b.abs().amax(2).clamp_min(AMAX_MIN)
    return (b * (FP8_MAX / a)[:, :, None]).view(M, H).to(torch.float8_e4m3fn), a / FP8_MAX


def _norm(s):
    r = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["residual_out"] = (r + s["residual"].float()).bfloat16()
        r = out["residual_out"].float()
    rstd = torch.rsqrt((r * r).mean(1) + EPS)
    y = r * rstd[:, None] * s["weight"]
    if s["y"] is not None:
        out["y"] = y.bfloat16()
    if s["rows"] is not None:
        out["codes"], out["scales"] = _quantise(y)
    if s["rstd"] is not None:
        out["rstd"] = rstd
    return out


def _norm_back(s):
    h = s["x"].float() * s["rstd"][:, None]
    dy = s["grad_y"].float()
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - h * (g * h).mean(1, keepdim=True))
    if s["grad_residual"] is not None:
        dx = dx + s["grad_residual"].float()
    return {"grad_x": dx.bfloat16(), "grad_weight": (dy * h).sum(0, dtype=torch.float64).float()}


def _route(s):
    c, logits = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    keep = torch.ones(T, dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"] != 0
    l = torch.where(keep[:, None], logits.float(), 0.0)
    v, idx = torch.sort(l, dim=1, descending=True, stable=True)   # ties go to the lowest expert
    v, idx = v[:, :k], idx[:, :k]
    top = v[:, :1]
    total = torch.exp(l - top).sum(1, keepdim=True)
    e = torch.exp(v - top)
    w = e / (e.sum(1, keepdim=True) if c["mode"] == RENORM else total)
    out = {"idx": torch.where(keep[:, None], idx, -1).int(), "w": torch.where(keep[:, None], w, 0.0)}
    if c["balance"]:
        lse = top + torch.log(total)
        p = torch.where(keep[:, None], torch.exp(l - lse), 0.0).sum(0, dtype=torch.float64)
        counts = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
        counts.index_add_(0, out["idx"].view(-1) + 1, torch.ones(T * k, dtype=torch.int32, device=l.device))
        out["counts"] = counts[1:]
        out["kept"] = keep.sum(dtype=torch.int32).view(1)
        n = out["kept"].double().clamp_min(1.0)
        out["loss"] = (E * (counts[1:] * p).sum() / (n * n * k)).float()
        out["lse"] = torch.where(keep, lse[:, 0], 0.0)
    return out


def _route_back(s):
    c, logits = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    keep = torch.ones(T, dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"] != 0
    l = torch.where(keep[:, None], logits.float(), 0.0)
    p = torch.exp(l - s["lse"][:, None])
    n = s["kept"].float().clamp_min(1.0)
    d = s["grad_loss"] * E * s["counts"] / (n * n * k)   # of the loss, by each expert's probability
    dl = p * (d - (p * d).sum(1, keepdim=True))
    gw = s["grad_w"] * s["w"]
    total = gw.sum(1, keepdim=True)
    if c["mode"] == RENORM:
        gw = gw - s["w"] * total
    else:
        dl = dl - p * total
    dl = dl.scatter_add(1, s["idx"].clamp_min(0).long(), gw)
    return {"grad_logits": torch.where(keep[:, None], dl, 0.0).to(logits.dtype)}


def _grouped(s, x, codes, scales):
    """Each row of x times its expert's weights, in float; rows without an expert: zero."""
    c = s["case"]
    G, M = c["G"], c["M"]
    _, width, K = codes.shape
    row = torch.arange(M, device="cuda", dtype=torch.int32)
    g = torch.searchsorted(s["offset"], row, right=True) - 1   # G: behind the last expert's rows
    at = (row - s["offset"][g]).long()
    a = torch.zeros(G + 1, s["most"], K, device="cuda")
    a[g, at] = x
    w = codes.float().view(G, width, K // BLOCK, BLOCK)
    w = (w * scales.repeat_interleave(BLOCK, 1)[:, :width, :, None]).view(G, width, K)
    y = torch.bmm(a[:G], w.transpose(1, 2).contiguous())[g.clamp_max(G - 1), at]
    return torch.where((g < G)[:, None], y, 0.0)


def _floats(codes, scales):
    M, K = codes.shape
    return (codes.float().view(M, K // BLOCK, BLOCK) * scales[:, :, None]).view(M, K)


def _product(s):
    K = s["case"]["K"]
    x = _floats(s["rows"][:, :K].view(torch.float8_e4m3fn), s["rows"][:, K:K + K // 32].view(torch.float32))
    return {"out": _grouped(s, x, s["codes"], s["scales"]).bfloat16()}


def _experts(s):
    H, F = s["case"]["H"], s["case"]["F"]
    x = _floats(s["rows"][:, :H].view(torch.float8_e4m3fn), s["rows"][:, H:H + H // 32].view(torch.float32))
    y = _grouped(s, x, s["codes"], s["scales"])
    gate, up = y[:, :F], y[:, F:]
    inner = _floats(*_quantise(gate / (1.0 + torch.exp(-gate)) * up))
    return {"out": _grouped(s, inner, s["codes2"], s["scales2"]).bfloat16()}


# ---- the operators by the library -------------------------------------------------------------------------------


def _own(s):
    import combine_topk_rank_amd as ep
    c = s["case"]
    op = c["op"]
    if op == "norm":
        ep.ep_rmsnorm(s["x"], s["residual"], s["weight"], EPS, s["residual_out"], s["y"], s["rows"], s["rstd"])
        out = {k: s[k] for k in ("residual_out", "y", "rstd") if s[k] is not None}
        return {**out, **_values(s["rows"], c["H"])} if s["rows"] is not None else out
    if op == "norm_back":
        ep.ep_rmsnorm_backward(s["x"], s["weight"], s["rstd"], s["grad_y"], s["grad_residual"], s["grad_x"],
                               s["grad_weight"], s["workspace"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"]}
    if op == "route":
        ep.ep_route(s["logits"], s["mask"], c["mode"], s["idx"], s["w"], s["counts"], s["kept"], s["lse"], s["loss"],
                    s["workspace"])
        out = {"idx": s["idx"], "w": s["w"]}
        if c["balance"]:
            out.update(counts=s["counts"], kept=s["kept"], lse=s["lse"], loss=s["loss"])
        return out
    if op == "route_back":
        ep.ep_route_backward(s["logits"], s["mask"], c["mode"], s["idx"], s["w"], s["counts"], s["kept"], s["lse"],
                             s["grad_w"], s["grad_loss"], s["grad_logits"])
        return {"grad_logits": s["grad_logits"]}
    if op == "product":
        ep.ep_expert_product(s["rows"], s["offset"], s["codes"], s["scales"], s["out"], s["status"])
    else:
        ep.ep_expert_gate_up(s["rows"], s["offset"], s["codes"], s["scales"], s["inner"], s["status"])
        ep.ep_expert_product(s["inner"], s["offset"], s["codes2"], s["scales2"], s["out"], s["status"])
    return {"out": s["out"]}


def _values(rows, H):
    """The codes and scales of 8-bit rows, as the numbers that they are (views)."""
    return {"codes": rows[:, :H].view(torch.float8_e4m3fn), "scales": rows[:, H:H + H // 32].view(torch.float32)}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "norm_back": _norm_back, "route": _route, "route_back": _route_back, "product": _product,
            "experts": _experts}[state["case"]["op"]](state)


# ---- the operators in 64 bits -----------------------------------------------------------------------------------


def _exact_rows(v):
    """What codes and scales of v would be if a code could hold any number."""
    b = v.unflatten(1, (-1, BLOCK))
    scale = torch.clamp(torch.linalg.vector_norm(b, ord=math.inf, dim=2), min=AMAX_MIN) / FP8_MAX
    return {"codes": (b / scale.unsqueeze(2)).flatten(1), "scales": scale}


def _exact_router(s):
    """The choices' gates and the balance loss as functions of logits in 64 bits, over the tokens that count."""
    c = s["case"]
    keep = torch.arange(c["T"], device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0]
    l = s["logits"][keep].double().requires_grad_(True)
    p = torch.softmax(l, 1)
    # a double holds a logit and, below it, its expert's number: no two are alike, and the lower expert is the larger
    order = (l.detach() - torch.arange(c["E"], device="cuda") * 1e-14).argsort(1, descending=True)[:, :c["k"]]
    w = p.gather(1, order)
    if c["mode"] == RENORM:
        w = w / w.sum(1, keepdim=True)
    share = torch.bincount(order.reshape(-1), minlength=c["E"]).double() / max(1, order.numel())
    return keep, l, w, c["E"] * (share * p.sum(0) / max(1, len(keep))).sum()


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm":
        r = s["x"].double()
        out = {}
        if s["residual"] is not None:
            r = r + s["residual"].double()
            out["residual_out"] = r
            r = r.bfloat16().double()
        rms = torch.sqrt(torch.linalg.vector_norm(r, dim=1) ** 2 / c["H"] + EPS)
        y = r / rms[:, None] * s["weight"].double()
        if s["y"] is not None:
            out["y"] = y
        if s["rows"] is not None:
            out.update(_exact_rows(y))
        if s["rstd"] is not None:
            out["rstd"] = 1.0 / rms
        return out
    if op == "norm_back":
        x, w = s["x"].double().requires_grad_(True), s["weight"].double().requires_grad_(True)
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
        dx, dw = torch.autograd.grad(y, (x, w), s["grad_y"].double())
        return {"grad_x": dx if s["grad_residual"] is None else dx + s["grad_residual"].double(), "grad_weight": dw}
    if op in ("route", "route_back"):
        keep, l, w, loss = _exact_router(s)
        if op == "route":
            full = torch.zeros(c["T"], c["k"], dtype=torch.float64, device="cuda").index_copy(0, keep, w.detach())
            out = {"idx": None, "w": full}
            if c["balance"]:
                lse = torch.zeros(c["T"], dtype=torch.float64, device="cuda")
                out.update(counts=None, kept=None, loss=loss.detach(), lse=lse.index_copy(0, keep, torch.logsumexp(l, 1).detach()))
            return out
        total = (w * s["grad_w"][keep].double()).sum() + loss * s["grad_loss"][0].double()
        dl, = torch.autograd.grad(total, l)
        return {"grad_logits": torch.zeros(c["T"], c["E"], dtype=torch.float64, device="cuda").index_copy(0, keep, dl)}
    bounds = s["offset"].tolist()
    K = c["K"] if op == "product" else c["H"]
    y = torch.zeros(c["M"], s["out"].shape[1], dtype=torch.float64, device="cuda")
    for g in range(c["G"]):
        a, b = bounds[g], bounds[g + 1]
        if a == b:
            continue
        left = s["rows"][a:b, :K].view(torch.float8_e4m3fn).double()
        left *= s["rows"][a:b, K:K + K // 32].view(torch.float32).double().repeat_interleave(BLOCK, 1)
        first = left @ _exact_weights(s["codes"][g], s["scales"][g])
        if op == "product":
            y[a:b] = first
            continue
        inner = _exact_rows(torch.nn.functional.silu(first[:, :c["F"]]) * first[:, c["F"]:])
        inner = inner["codes"].to(torch.float8_e4m3fn).double() * inner["scales"].repeat_interleave(BLOCK, 1)
        y[a:b] = inner @ _exact_weights(s["codes2"][g], s["scales2"][g])
    return {"out": y}


def _exact_weights(codes, scales):
    """[K, N] of one expert."""
    N = codes.shape[0]
    return (codes.double() * scales.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)).t().contiguous()
