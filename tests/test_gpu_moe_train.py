"""The training pass of a block as a user runs it: BuffersMoETrain's forward and
backward, and the clipping of what comes out, against 64 bits.

The reference runs the block in 64 bits for the library's own choices and
differentiates it by itself.  The library rounds to bf16 on the way (rows, inner
rows, their gradients): each tensor's norm may be off by the roundings that led to
it, at most ten in a row, 2^-9 each on average: 2^-5.5."""

import pytest
import torch

from gpu_helpers import log

pytestmark = pytest.mark.gpu

EPS = 1e-6
OFF = 2.0 ** -5.5


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def make(T, H, E, F, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    return dict(x=f(T, H).bfloat16(), residual=(2 * f(T, H)).bfloat16(), weight=1 + 0.1 * f(H), router=(f(E, H) * H ** -0.5),
                w1=(f(E, 2 * F, H) * H ** -0.5).bfloat16(), w2=(f(E, H, F) * F ** -0.5).bfloat16(),
                grad_out=f(T, H).bfloat16(), grad_residual=f(T, H).bfloat16(), grad_loss=torch.full((1,), 3.0, device="cuda"))


def reference(d, idx, mask, mode, k, residual=True):
    """Outputs and gradients in 64 bits for the given choices."""
    leaf = {n: d[n].double().requires_grad_(True) for n in ("x", "weight", "router", "w1", "w2")}
    res = d["residual"].double() if residual else 0.0
    r = leaf["x"] + res
    h = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * leaf["weight"]
    p = torch.softmax(h @ leaf["router"].t(), 1)
    keep = torch.ones(len(h), dtype=torch.bool, device="cuda") if mask is None else mask != 0
    w = p.gather(1, idx.clamp_min(0).long()) * (idx >= 0)
    if mode == 1:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    E, F = d["w1"].shape[0], d["w2"].shape[2]
    out = torch.zeros_like(h)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            g = h[t] @ leaf["w1"][e].t()
            y = (torch.nn.functional.silu(g[:, :F]) * g[:, F:]) @ leaf["w2"][e].t()
            out = out.index_add(0, t, w[t, j, None] * y)
    n = keep.sum().clamp_min(1)
    counts = torch.bincount(idx[idx >= 0].long(), minlength=E).double()
    loss = E * (counts / (n * k) * p[keep].sum(0) / n).sum()
    total = (out * d["grad_out"].double()).sum() + loss * d["grad_loss"].double()[0] + (r * d["grad_residual"].double()).sum()
    return out, loss, dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))


def near(got, want, what, off=OFF):
    got, want = got.double(), want.detach()
    assert torch.isfinite(got).all(), what
    assert float((got - want).norm()) <= off * float(want.norm()) + 1e-12, (what, float((got - want).norm() / want.norm()))


CASES = [(1, 64, 8, 2, 2, 32, False, 1, True), (7, 128, 16, 4, 4, 64, False, 0, True), (128, 256, 16, 4, 2, 72, True, 1, True),
         (700, 512, 32, 8, 4, 128, True, 1, True), (500, 264, 6, 3, 3, 200, True, 0, False), (3000, 256, 8, 2, 2, 320, True, 1, True)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,E,R,k,F,masked,mode,residual", CASES)
def test_forward_and_backward(ep, T, H, E, R, k, F, masked, mode, residual, kind):
    log(f"[train block] T={T} H={H} E={E} k={k} F={F} mode={mode} {kind}")
    d = make(T, H, E, F, 1)
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.uint8, device="cuda")
        mask[::5] = 0
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, R, k), F, weights_dtype=kind)
    seen = {}

    def router(n):
        seen["n"] = n
        return n.float() @ d["router"].t()

    def router_backward(g):
        seen["grad"] = g.t() @ seen["n"].float()
        return (g @ d["router"]).bfloat16()

    out = buf.forward(d["x"], d["residual"] if residual else None, d["weight"], EPS, router, d["w1"], d["w2"], mode, mask)
    got_out, got_loss = out.clone(), buf.balance_loss.clone()
    grad_x = buf.backward(d["grad_out"], d["grad_residual"], d["grad_loss"], router_backward)
    assert int(buf.dev_status) == 0
    want, loss, grads = reference(d, buf.topk_idx, mask, mode, k, residual)
    near(got_out, want, "out")
    near(got_loss, loss.view(1), "loss")
    near(grad_x, grads["x"], "grad_x")
    near(buf.grad_weight, grads["weight"], "grad_weight")
    near(seen["grad"], grads["router"], "grad_router")
    near(buf.grad_gate_up, grads["w1"], "grad_gate_up")
    near(buf.grad_down, grads["w2"], "grad_down")
    assert buf.grad_gate_up.dtype is kind
    # an expert without a token has no gradient
    idle = torch.bincount(buf.topk_idx[buf.topk_idx >= 0].long(), minlength=E) == 0
    assert (buf.grad_gate_up[idle] == 0).all() and (buf.grad_down[idle] == 0).all()
    # clipped together with the router's
    grads = buf.gradients()
    s, n = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.zeros(ep.ep_grad_norm_workspace_bytes(grads), dtype=torch.uint8, device="cuda")
    before = [t.double().clone() for t in grads.tensors]
    ep.ep_grad_norm(grads, s, n, ws)
    norm = float(sum((t ** 2).sum() for t in before)) ** 0.5
    assert abs(float(n) - norm) <= 1e-6 * norm
    ep.ep_grad_clip(grads, s, 0.25 * norm)
    for t, b in zip((buf.grad_weight, buf.grad_gate_up, buf.grad_down), before):
        near(t, 0.25 * b, "clipped", 2.0 ** -8)


def test_backward_needs_its_forward(ep):
    T, H, E, F, k = 20, 64, 8, 32, 2
    d = make(T, H, E, F, 2)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F)
    with pytest.raises(RuntimeError):
        buf.backward(d["grad_out"])
    run = lambda: buf.forward(d["x"], None, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["w2"])  # noqa: E731
    run()
    first = buf.backward(d["grad_out"]).clone()
    with pytest.raises(RuntimeError):
        buf.backward(d["grad_out"])
    run()
    assert torch.equal(buf.backward(d["grad_out"]), first)      # the same bits again
    with pytest.raises(ValueError):
        ep.BuffersMoETrain(ep.shape(T, 128, E, 2, k, ep.EP_FMT_FP8_E4M3_B128), F)


def test_a_refused_backward_leaves_the_forward(ep):
    T, H, E, F, k = 20, 64, 8, 32, 2
    d = make(T, H, E, F, 2)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F)
    run = lambda: buf.forward(d["x"], None, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["w2"])  # noqa: E731
    run()
    first = buf.backward(d["grad_out"]).clone()
    run()
    with pytest.raises(ValueError):
        buf.backward(d["grad_out"][:-1])
    assert torch.equal(buf.backward(d["grad_out"]), first)


def test_captured(ep):
    """A whole step in a graph, replayed on other inputs with eager work between."""
    T, H, E, F, k = 300, 128, 16, 64, 4
    d = make(T, H, E, F, 3)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 4, k), F)
    router = d["router"].t().contiguous()
    s, n = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    grads, ws = buf.gradients(), torch.zeros(ep.ep_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def step():
        buf.forward(d["x"], d["residual"], d["weight"], EPS, lambda v: v.float() @ router, d["w1"], d["w2"])
        buf.backward(d["grad_out"], d["grad_residual"], d["grad_loss"], lambda g: (g @ d["router"]).bfloat16())
        ep.ep_grad_norm(grads, s, n, ws)
        ep.ep_grad_clip(grads, s, 1.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (buf.out, buf.grad_x, buf.grad_weight, buf.grad_gate_up, buf.grad_down, buf.balance_loss, n)
    for i in range(4):
        d["x"].copy_(torch.randn(T, H, device="cuda"))
        d["grad_out"].copy_(torch.randn(T, H, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
    assert int(buf.dev_status) == 0


def test_the_rank_layout_between_the_products(ep):
    """One row for each (token, rank), dispatched and combined per rank, its gates and
    rows differentiated: a rank's own function here is a scaling."""
    T, H, E, R, k = 200, 256, 32, 8, 4
    d = make(T, H, E, 64, 4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.rand(T, E, device="cuda", generator=gen).argsort(1)[:, :k].int().contiguous()
    w = torch.rand(T, k, device="cuda", generator=gen)
    s = ep.shape(T, H, E, R, k)
    buf = ep.Buffers(s)
    buf.layout(idx)
    buf.dispatch(d["x"], idx, w)
    P = int(buf.rank_offset[-1])
    sent = buf.send_buf.view(torch.bfloat16)
    scale = 2.0 ** torch.randint(-1, 2, (buf.capacity_rows, 1), device="cuda", generator=gen).float()
    y = (sent.float() * scale).bfloat16()
    y[P:] = 0
    buf.combine(y, idx, w)
    grad_y, grad_w, grad_x = torch.zeros_like(y), torch.empty_like(w), torch.empty_like(d["x"])
    ep.ep_combine_backward(s, y, idx, w, buf.send_slot, d["grad_out"], grad_y, grad_w, buf.dev_status)
    ep.ep_dispatch_backward(s, idx, buf.send_slot, (grad_y.float() * scale).bfloat16(), None, None, grad_x, None, buf.dev_status)
    assert int(buf.dev_status) == 0
    x64, w64 = d["x"].double().requires_grad_(True), w.double().requires_grad_(True)
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for r in range(R):
        has = buf.send_slot[:, r] >= 0
        weight = (w64 * (torch.div(idx, E // R, rounding_mode="floor") == r)).sum(1)
        out = out + torch.where(has[:, None], weight[:, None] * scale[buf.send_slot[:, r].clamp_min(0).long()].double() * x64, 0.0)
    near(buf.out, out, "out", 2.0 ** -8)
    gx, gw = torch.autograd.grad(out, (x64, w64), d["grad_out"].double())
    near(grad_x, gx, "grad_x", 2.0 ** -7)
    near(grad_w, gw, "grad_w", 1e-5)


def test_a_forward_that_ends_early_leaves_no_forward(ep):
    """Its buffers hold parts of two steps then: no backward may take them for one."""
    T, H, E, F, k = 20, 64, 8, 32, 2
    d = make(T, H, E, F, 2)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F)
    router = lambda n: n.float() @ d["router"].t()  # noqa: E731
    run = lambda x=d["x"], r=router, w2=d["w2"]: buf.forward(x, None, d["weight"], EPS, r, d["w1"], w2)  # noqa: E731
    run()
    first = buf.backward(d["grad_out"]).clone()

    def no_router(n):
        raise KeyError("router")

    for kind, bad in ((KeyError, dict(r=no_router)), (ValueError, dict(w2=d["w2"].float())), (ValueError, dict(x=d["x"].float())),
                      (ValueError, dict(r=lambda n: router(n)[:, :4]))):
        run()
        with pytest.raises(kind):
            run(**bad)
        with pytest.raises(RuntimeError, match="forward"):
            buf.backward(d["grad_out"])
    run()
    assert torch.equal(buf.backward(d["grad_out"]), first)


def test_a_backward_refused_for_any_gradient_leaves_the_forward(ep):
    T, H, E, F, k = 20, 64, 8, 32, 2
    d = make(T, H, E, F, 2)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F)
    run = lambda: buf.forward(d["x"], None, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["w2"])  # noqa: E731
    good = dict(grad_out=d["grad_out"], grad_residual=d["grad_residual"], grad_balance_loss=d["grad_loss"])
    run()
    first = buf.backward(**good).clone()
    run()
    for name, t in good.items():
        for bad in (t.double(), t[:0], t.cpu(), torch.cat([t, t])):
            with pytest.raises(ValueError, match=name):
                buf.backward(**{**good, name: bad})
    with pytest.raises(ValueError, match="grad_residual"):
        buf.backward(**{**good, "grad_residual": torch.zeros(H, T, dtype=torch.bfloat16, device="cuda").t()})
    assert torch.equal(buf.backward(**good), first)
    # the router's part comes when the forward's values have become their gradients
    run()
    with pytest.raises(ValueError, match="grad_other"):
        buf.backward(**good, router_backward=lambda g: g)
    with pytest.raises(RuntimeError, match="forward"):
        buf.backward(**good)


def test_an_input_of_autograd(ep):
    """x may be a tensor that autograd follows, as an embedding's: the buffers take no part in it."""
    T, H, E, F, k = 20, 64, 8, 32, 2
    d = make(T, H, E, F, 2)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F)
    table = d["x"].clone().requires_grad_(True)
    for residual in (None, d["residual"]):
        for _ in range(2):
            x = table * 1.0
            out = buf.forward(x, residual, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["w2"])
            assert not any(t.requires_grad for t in (out, buf.residual, buf.normed)) and buf.residual.grad_fn is None
            x.backward(buf.backward(d["grad_out"]))
        assert torch.isfinite(table.grad).all()


# no token; one; a mask that leaves none
@pytest.mark.parametrize("T,masked", [(0, False), (1, True), (40, True)])
def test_a_block_without_rows(ep, T, masked):
    """No expert has a row: no output, no gradient but what goes past the block."""
    H, E, F, k = 64, 8, 32, 2
    d = make(T, H, E, F, 6)
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda") if masked else None
    for kind in (torch.bfloat16, torch.float32):
        buf = ep.BuffersMoETrain(ep.shape(T, H, E, 2, k), F, weights_dtype=kind)
        for t in (buf.grad_gate_up, buf.grad_down, buf.grad_weight, buf.out, buf.y, buf.pre):
            t.fill_(float("nan"))
        out = buf.forward(d["x"], d["residual"], d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["w2"], token_mask=mask)
        assert out.shape == (T, H) and (out == 0).all() and float(buf.balance_loss) == 0.0
        grad_x = buf.backward(d["grad_out"], d["grad_residual"], d["grad_loss"], lambda g: (g @ d["router"]).bfloat16())
        assert int(buf.dev_status) == 0
        assert torch.equal(grad_x, d["grad_residual"])
        for t in (buf.grad_gate_up, buf.grad_down, buf.grad_weight):
            assert (t == 0).all()
        s, n = torch.ones(1, dtype=torch.float64, device="cuda"), torch.ones(1, device="cuda")
        ep.ep_grad_norm(buf.gradients(), s, n, torch.zeros(ep.ep_grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda"))
        assert float(n) == 0.0


@pytest.mark.parametrize("T,H,E,k,F,takes", [(1024, 264, 256, 8, 72, "ss"), (4096, 1024, 256, 8, 520, "BB")])
def test_a_block_of_256_experts(ep, T, H, E, k, F, takes):
    """More experts than a wavefront has lanes, about T k / E rows each, through small and big tiles."""
    d = make(T, H, E, F, 7)
    buf = ep.BuffersMoETrain(ep.shape(T, H, E, 32, k), F)
    plans = [ep.ep_expert_bf16_plan(p, E, T * k, 2 * F, H) for p in (ep.EP_PRODUCT_GATE_UP, ep.EP_PRODUCT_ROWS_BACKWARD)]
    assert "".join("B" if p == ep.EP_TILES_BIG else "s" for p in plans) == takes
    seen = {}

    def router(n):
        seen["n"] = n
        return n.float() @ d["router"].t()

    out = buf.forward(d["x"], d["residual"], d["weight"], EPS, router, d["w1"], d["w2"])
    got_out, got_loss = out.clone(), buf.balance_loss.clone()
    grad_x = buf.backward(d["grad_out"], d["grad_residual"], d["grad_loss"], lambda g: (g @ d["router"]).bfloat16())
    assert int(buf.dev_status) == 0
    want, loss, grads = reference(d, buf.topk_idx, None, 1, k)
    near(got_out, want, "out")
    near(got_loss, loss.view(1), "loss")
    near(grad_x, grads["x"], "grad_x")
    near(buf.grad_weight, grads["weight"], "grad_weight")
    near(buf.grad_gate_up, grads["w1"], "grad_gate_up")
    near(buf.grad_down, grads["w2"], "grad_down")
