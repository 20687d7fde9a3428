"""The bf16 expert products as they are called: their own forward differenced, and calls
whose weights' gradient is summed in parts through a workspace, on two streams and in a
graph, with big and with small tiles."""

import pytest
import torch

import training_refs as X
from test_gpu_expert_bf16 import BF, POISON, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def tiles(ep, c):
    return "".join("B" if ep.ep_expert_bf16_plan(p, c.G, c.M, c.N, c.K) == ep.EP_TILES_BIG else "s" for p in range(4) if p != 1)


def ones(c, *shape):
    return torch.randint(-1, 2, shape, device="cuda", generator=c.gen).bfloat16()


@pytest.mark.parametrize("sizes,N,K,takes", [([40, 0, 25], 72, 120, "ssB"), ([20000], 2064, 120, "BsB"), ([20000], 120, 2064, "sBB")])
def test_differences_of_the_products_own_forward(ep, sizes, N, K, takes):
    """Central differences of ep_expert_product_bf16 against its gradients, in a direction for
    the rows and one for the weights.

    All operands are -1, 0 or 1, so rows and weights with the step added or taken away are
    -2 to 2.  With K <= 120 every output is a whole number up to 240 and exact in bf16; so is the
    rows' gradient with N <= 120.  The longer products have 64 values other than 0 in a row (and,
    for the rows' gradient, in a column), so that the same holds.  The weights' gradient is taken
    in float.  Each side is a whole number below 2^53: the two are equal."""
    c = Case(sizes, N, K, whole=True, seed=31)
    assert tiles(ep, c) == takes
    M, G = c.M, c.G
    c.rows, c.w, c.grad_out = ones(c, M, K), ones(c, G, N, K), ones(c, M, N)
    step_r, step_w = ones(c, M, K), ones(c, G, N, K)
    if K > 120:
        for t in (c.rows, step_r):
            t[:, 64:] = 0
    if N > 120:
        c.grad_out[:, 64:] = 0
    gr, gw = torch.zeros(M, K, **BF), torch.zeros(G, N, K, device="cuda")
    ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, c.workspace(ep))

    def f(rows, w):
        out = torch.zeros(M, N, **BF)
        ep.ep_expert_product_bf16(rows, c.off, w, out, c.st)
        assert float(out.abs().max()) <= 256
        return out.double()

    assert float(gr.abs().max()) <= 256
    d = c.grad_out.double()
    by_rows = (d * (f(c.rows + step_r, c.w) - f(c.rows - step_r, c.w))).sum() / 2
    by_w = (d * (f(c.rows, c.w + step_w) - f(c.rows, c.w - step_w))).sum() / 2
    assert by_rows == (gr.double() * step_r.double()).sum() != 0
    assert by_w == (gw.double() * step_w.double()).sum() != 0
    assert int(c.st) == 0


def test_differences_of_the_gates_own_forward(ep):
    """Central differences of ep_expert_gate_up_bf16 against the weights' gradient that its
    backward makes.

    A row of rows is one at its own c, so out[m, f] = silu(w[f, m]) * w[F + f, m] and each weight
    reaches one output.  Gates -1 to 4, ups 1/2 to 2 and the step h = 1/4 are exact in bf16.
    Each output is rounded once (2^-8) after a few float operations (8 * 2^-24 * 4); the weights'
    gradient is that of a grad_pre rounded once.  Along an up the output is linear; along a
    gate the quotient is off by h^2 / 6 * max |silu'''| * up, and |silu'''| = |3 s'' + g s'''| <=
    3 * 0.0963 + 4.25 * 0.125 = 0.83 (s'' and s''' the sigmoid's, at gates up to 4.25)."""
    F, K, h = 72, 64, 0.25
    g = torch.Generator(device="cuda").manual_seed(32)
    eighths = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, device="cuda", generator=g) / 8  # noqa: E731
    w = torch.cat([eighths(-8, 32, 1, F, K), eighths(4, 16, 1, F, K)], 1).bfloat16()
    rows = torch.eye(K, **BF)
    d = (0.5 + eighths(0, 8, K, F)).bfloat16()
    off, st = torch.tensor([0, K], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def f(w):
        out = torch.zeros(K, F, **BF)
        ep.ep_expert_gate_up_bf16(rows, off, w, None, out, st)
        return out.double()

    pre, out = torch.zeros(K, 2 * F, **BF), torch.zeros(K, F, **BF)
    ep.ep_expert_gate_up_bf16(rows, off, w, pre, out, st)
    assert torch.equal(pre, w[0].t())
    gp, gw = torch.zeros(K, 2 * F, **BF), torch.zeros(1, 2 * F, K, device="cuda")
    ep.ep_expert_gate_up_bf16_backward(rows, off, w, pre, d, gp, None, gw, st,
                                       torch.empty(max(16, ep.ep_expert_backward_workspace_bytes(1, K, 2 * F, K)), dtype=torch.uint8, device="cuda"))
    assert torch.equal(gw[0], gp.t().float())
    once = X.U_BF16 + 32 * X.U32
    for part in (slice(0, F), slice(F, 2 * F)):
        step = torch.zeros_like(w)
        step[:, part] = h
        up, down = f(w + step), f(w - step)
        quotient = d.double() * (up - down) / (2 * h)
        off_by = d.double() * once * (up.abs() + down.abs()) / (2 * h) * (1 + once)
        if part.start == 0:
            off_by = off_by + d.double() * h * h / 6 * 0.83 * w[0, F:].t().double()
        got = gw[0, part].t().double()
        assert ((got - quotient).abs() <= off_by + got.abs() * once).all()
        # all together: much nearer than a factor or the other half would be
        assert float((got - quotient).sum().abs() / quotient.sum()) <= 0.02
    assert int(st) == 0


SPLIT = [([5000, 0, 9000], 264, 520, "ssB"), ([9000, 5000], 1040, 520, "BBB")]


@pytest.mark.parametrize("sizes,N,K,takes", SPLIT)
def test_two_streams_with_sums_in_parts(ep, sizes, N, K, takes):
    """Two backward calls at once, on streams of their own, each with its own workspace."""
    cases = [Case(s, N, K, whole=True, seed=33 + i) for i, s in enumerate((sizes, sizes[::-1]))]
    outs = [(torch.full((c.M, K), POISON, **BF), torch.full((c.G, N, K), POISON, device="cuda"), c.workspace(ep)) for c in cases]
    assert all(tiles(ep, c) == takes and ws is not None for c, (_, _, ws) in zip(cases, outs))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, (gr, gw, ws), s in zip(cases, outs, (None, side)):
            ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, ws, s)
    torch.cuda.synchronize()
    for c, (gr, gw, _) in zip(cases, outs):
        c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), N, "grad_rows")
        c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), max(sizes), "grad_w")
        assert int(c.st) == 0


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,N,K,takes", [([5000, 0, 9000], 528, 136, "ssB"), ([9000, 0, 5000], 2064, 520, "BBB")])
def test_captured_with_sums_in_parts(ep, sizes, N, K, takes, kind):
    """Gate, product and both backward calls in one graph, replayed on other inputs and offsets
    with the program's own work between."""
    c = Case(sizes, N, K, seed=34)
    F, M = N // 2, c.M
    down = Case(sizes, K, F, seed=35)          # the second product, from the gate's outputs
    assert tiles(ep, c) == takes
    ws, ws2 = c.workspace(ep), down.workspace(ep)
    assert ws is not None and ws2 is not None
    c.w *= K ** -0.5
    down.w *= F ** -0.5
    pre, inner, out = torch.zeros(M, N, **BF), torch.zeros(M, F, **BF), torch.zeros(M, K, **BF)
    gi, gp, gr = torch.zeros(M, F, **BF), torch.zeros(M, N, **BF), torch.zeros(M, K, **BF)
    gw, gw2 = torch.zeros(c.G, N, K, dtype=kind, device="cuda"), torch.zeros(c.G, K, F, dtype=kind, device="cuda")

    def step():
        ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre, inner, c.st)
        ep.ep_expert_product_bf16(inner, c.off, down.w, out, c.st)
        ep.ep_expert_product_bf16_backward(inner, c.off, down.w, down.grad_out, gi, gw2, c.st, ws2)
        ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, pre, gi, gp, gr, gw, c.st, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    a, b = sizes[0], M
    for i, off in enumerate(([0, a, a, b], [0, 1, b - 1, b], [0, 0, 0, b], [10, 300, a, b - 20])):
        c.off.copy_(torch.tensor(off, dtype=torch.int32))
        c.rows.copy_(c.values(M, K))
        outs = (pre, inner, out, gi, gp, gr, gw, gw2)
        for t in outs:
            t.fill_(POISON)
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(POISON)
        ws.fill_(0xFF)
        ws2.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want)), i
        assert all(torch.isfinite(t.float()).all() for t in outs)
    assert int(c.st) == 0


@pytest.mark.parametrize("rows,takes", [(70, "ssB"), (6000, "BBB")])
def test_far_weights(ep, rows, takes):
    """Weights whose bytes lie beyond 2^32: 40 experts of 8192 x 8192, 5.4 GB, rows at two of them."""
    G, N, K = 40, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(36)
    whole = lambda *s: torch.randint(-2, 3, s, device="cuda", generator=g).bfloat16()  # noqa: E731
    w = torch.zeros(G, N, K, **BF)
    w[0], w[G - 1] = whole(N, K), whole(N, K)
    M = 3 + rows
    off = torch.tensor([0] + [3] * (G - 1) + [M], dtype=torch.int32, device="cuda")
    x, d, st = whole(M, K), whole(M, N), torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = [ep.ep_expert_bf16_plan(p, G, M, N, K) for p in (ep.EP_PRODUCT_FORWARD, ep.EP_PRODUCT_ROWS_BACKWARD, ep.EP_PRODUCT_WEIGHTS_BACKWARD)]
    assert "".join("B" if p == ep.EP_TILES_BIG else "s" for p in plan) == takes
    out, gr, gw = torch.full((M, N), POISON, **BF), torch.full((M, K), POISON, **BF), torch.full((G, N, K), POISON, **BF)
    ep.ep_expert_product_bf16(x, off, w, out, st)
    n = ep.ep_expert_backward_workspace_bytes(G, M, N, K)
    ep.ep_expert_product_bf16_backward(x, off, w, d, gr, gw, st, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    assert int(st) == 0
    for e, a, b in ((0, 0, 3), (G - 1, 3, M)):      # every sum below 2^24: exact in float
        assert torch.equal(out[a:b].double(), (x[a:b].double() @ w[e].double().t().contiguous()).bfloat16().double())
        assert torch.equal(gr[a:b].double(), (d[a:b].double() @ w[e].double()).bfloat16().double())
        assert torch.equal(gw[e].double(), (d[a:b].double().t().contiguous() @ x[a:b].double()).bfloat16().double())
    assert (gw[1:G - 1] == 0).all()


@pytest.mark.parametrize("rows,N", [(300, 72), (9000, 2056)])
def test_far_rows(ep, rows, N):
    """Rows whose bytes lie beyond 2^32: the last ones of 300 000 x 8192, 4.9 GB."""
    M, K = 300_000, 8192
    g = torch.Generator(device="cuda").manual_seed(37)
    whole = lambda *s: torch.randint(-2, 3, s, device="cuda", generator=g).bfloat16()  # noqa: E731
    x, d, w = torch.zeros(M, K, **BF), torch.zeros(M, N, **BF), whole(2, N, K)
    a = M - rows
    x[a:], d[a:] = whole(rows, K), whole(rows, N)
    off, st = torch.tensor([a, a + 100, M], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, gr, gw = torch.full((M, N), POISON, **BF), torch.full((M, K), POISON, **BF), torch.full((2, N, K), POISON, device="cuda")
    ep.ep_expert_product_bf16(x, off, w, out, st)
    n = ep.ep_expert_backward_workspace_bytes(2, M, N, K)
    ep.ep_expert_product_bf16_backward(x, off, w, d, gr, gw, st, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None)
    assert int(st) == 0
    assert (out[:a] == POISON).all() and (gr[:a] == POISON).all()
    for e, lo, hi in ((0, a, a + 100), (1, a + 100, M)):
        assert torch.equal(out[lo:hi].double(), (x[lo:hi].double() @ w[e].double().t().contiguous()).bfloat16().double())
        assert torch.equal(gr[lo:hi].double(), (d[lo:hi].double() @ w[e].double()).bfloat16().double())
        assert torch.equal(gw[e].double(), d[lo:hi].double().t().contiguous() @ x[lo:hi].double())
