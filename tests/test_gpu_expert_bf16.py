"""The bf16 expert products and their gradients against 64 bits.

Two kinds of inputs.  Small whole numbers: every product and sum is exact in
float, so the result is bit for bit the rounded 64-bit one; a row, column or
block that goes astray shows at once.  Random ones: within training_refs.SUM of
the magnitudes' sum, and the output's rounding."""

import pytest
import torch

import training_refs as X
from gpu_helpers import log
from operator_refs import assert_close

pytestmark = pytest.mark.gpu

POISON = -99.0
BF = dict(dtype=torch.bfloat16, device="cuda")


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


class Case:
    def __init__(self, sizes, N, K, first=0, behind=0, whole=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.G, self.N, self.K, self.gen = len(sizes), N, K, g
        self.M = first + sum(sizes) + behind
        self.off = X.spread(sizes, self.M, first)
        self.whole = whole
        self.rows, self.w = self.values(self.M, K), self.values(self.G, N, K)
        self.grad_out = self.values(self.M, N)
        self.inside = torch.zeros(self.M, dtype=torch.bool, device="cuda")
        self.inside[first:first + sum(sizes)] = True
        # what no expert has is never read into a result
        self.rows[~self.inside] = float("nan")
        self.grad_out[~self.inside] = float("nan")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def values(self, *shape):
        if self.whole:
            return torch.randint(-3, 4, shape, device="cuda", generator=self.gen).bfloat16()
        return torch.randn(*shape, device="cuda", generator=self.gen).bfloat16()

    def workspace(self, ep, fill=0xFF):
        n = ep.ep_expert_backward_workspace_bytes(self.G, self.M, self.N, self.K)
        return torch.full((n,), fill, dtype=torch.uint8, device="cuda") if n else None

    def check(self, got, want, mag, n, what):
        """Rows of an output [M, ...]: those of an expert right, the others as they were."""
        assert (got[~self.inside] == POISON).all(), what
        self.close(got[self.inside], want[self.inside], mag[self.inside], n, what)

    def close(self, got, want, mag, n, what):
        if self.whole:
            assert float(mag.max() if mag.numel() else 0) < 2 ** 24
            assert torch.equal(got, want.to(got.dtype)), what
        elif got.dtype == torch.float32:
            assert_close(got, want, mag * X.SUM(n), what)
        else:
            assert_close(got, want, X.bf16_tol(want, mag * X.SUM(n)), what)


# sizes of the groups, N, K, rows before the first group and behind the last
SHAPES = [
    ([1], 8, 8, 0, 0), ([1], 64, 64, 0, 0), ([3], 16, 72, 2, 1), ([64], 64, 64, 0, 0), ([65], 72, 136, 0, 3),
    ([0, 5, 0, 0, 70, 1], 200, 264, 7, 9), ([1] * 8, 520, 328, 0, 0), ([31, 128, 2, 63], 136, 1000, 0, 5),
    ([0, 0], 64, 128, 4, 4), ([17] * 70, 40, 48, 1, 1), ([256, 300], 512, 256, 0, 0), ([700, 0, 33], 264, 520, 3, 0),
    ([1000], 1032, 200, 0, 1), ([2, 2000, 1], 24, 2056, 0, 0), ([5, 9], 2048, 24, 0, 0),
]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("sizes,N,K,first,behind", SHAPES)
def test_product(ep, sizes, N, K, first, behind, whole):
    log(f"[bf16 product] {sizes[:6]} N={N} K={K} whole={whole}")
    c = Case(sizes, N, K, first, behind, whole)
    out = torch.full((c.M, N), POISON, **BF)
    ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
    assert int(c.st) == 0
    c.check(out, *X.product64(c.rows, c.off, c.w), K, "out")


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("sizes,N,K,first,behind", SHAPES)
def test_product_backward(ep, sizes, N, K, first, behind, whole, kind):
    log(f"[bf16 product back] {sizes[:6]} N={N} K={K} whole={whole} {kind}")
    c = Case(sizes, N, K, first, behind, whole, seed=1)
    grad_rows = torch.full((c.M, K), POISON, **BF)
    grad_w = torch.full((c.G, N, K), POISON, dtype=kind, device="cuda")
    ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, grad_rows, grad_w, c.st, c.workspace(ep))
    assert int(c.st) == 0
    c.check(grad_rows, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), N, "grad_rows")
    c.close(grad_w, *X.weights64(c.rows, c.off, c.grad_out), max(sizes), "grad_w")
    # each alone, from what it needs alone
    r, w = torch.full_like(grad_rows, POISON), torch.full_like(grad_w, POISON)
    ep.ep_expert_product_bf16_backward(None, c.off, c.w, c.grad_out, r, None, c.st)
    ep.ep_expert_product_bf16_backward(c.rows, c.off, None, c.grad_out, None, w, c.st, c.workspace(ep, 0))
    assert torch.equal(r, grad_rows) and torch.equal(w, grad_w) and int(c.st) == 0


@pytest.mark.parametrize("rows_at,w_at", [(0, 1), (3, 0), (7, 7), (1, 4), (5, 2)])
@pytest.mark.parametrize("K", [8, 56, 64, 72, 256, 328, 520])
def test_operands_off_lines(ep, rows_at, w_at, K):
    """Tensors that begin 16 bytes times rows_at and w_at behind a line, NaN around them."""
    log(f"[bf16 product off lines] rows {rows_at} w {w_at} K={K}")
    c = Case([3, 0, 66, 17], 80, K, whole=True, seed=13)

    def moved(x, at):
        room = torch.full((x.numel() + 192,), float("nan"), **BF)
        room = room[-room.data_ptr() % 128 // 2:]
        y = room[8 * at:][:x.numel()].view(x.shape)
        assert y.data_ptr() % 128 == 16 * at
        return y.copy_(x)

    rows, w, grad_out = moved(c.rows, rows_at), moved(c.w, w_at), moved(c.grad_out, w_at)
    out, grad_rows = torch.full((c.M, c.N), POISON, **BF), torch.full((c.M, K), POISON, **BF)
    grad_w, h, pre = torch.full_like(w, POISON), torch.full((c.M, 40), POISON, **BF), torch.full((c.M, 80), POISON, **BF)
    ep.ep_expert_product_bf16(rows, c.off, w, out, c.st)
    ep.ep_expert_product_bf16_backward(rows, c.off, w, grad_out, grad_rows, grad_w, c.st, c.workspace(ep))
    ep.ep_expert_gate_up_bf16(rows, c.off, w, pre, h, c.st)
    assert int(c.st) == 0
    c.check(out, *X.product64(c.rows, c.off, c.w), K, "out")
    c.check(grad_rows, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), c.N, "grad_rows")
    c.close(grad_w, *X.weights64(c.rows, c.off, c.grad_out), 66, "grad_w")
    c.check(pre, *X.product64(c.rows, c.off, c.w), K, "pre")


GATES = [([1], 8, 8, 0, 0), ([3], 24, 72, 2, 1), ([64], 32, 64, 0, 0), ([65], 40, 136, 0, 3), ([0, 5, 0, 0, 70, 1], 200, 264, 7, 9),
         ([1] * 8, 520, 328, 0, 0), ([31, 128, 2, 63], 136, 1000, 0, 5), ([0, 0], 64, 128, 4, 4), ([17] * 70, 40, 48, 1, 1),
         ([300, 256], 256, 512, 0, 0), ([700, 0, 33], 264, 520, 3, 0)]


def gate64(pre, off_pre):
    """silu(gate) * up of 64-bit pre, and how far off values make it."""
    F = pre.shape[1] // 2
    g, u = pre[:, :F], pre[:, F:]
    s = torch.sigmoid(g)
    h = g * s * u
    # silu' <= 1.1; the sigmoid's exp, sum, quotient and two products: eight roundings.  A
    # sigmoid below float's normal range (a gate below -87.3) is held in steps of 2^-149: the
    # product is off by one of them times |g u|
    return h, (g * u).abs() * 2.0 ** -149 + 1.1 * off_pre[:, :F] * u.abs() + (g * s).abs() * off_pre[:, F:] + 1.1 * off_pre[:, :F] * off_pre[:, F:] + 8 * X.U32 * h.abs() * 4


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("sizes,F,K,first,behind", GATES)
def test_gate_up(ep, sizes, F, K, first, behind, keep):
    log(f"[bf16 gate up] {sizes[:6]} F={F} K={K}")
    c = Case(sizes, 2 * F, K, first, behind)
    c.w *= K ** -0.5
    out, pre = torch.full((c.M, F), POISON, **BF), torch.full((c.M, 2 * F), POISON, **BF)
    ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre if keep else None, out, c.st)
    assert int(c.st) == 0
    want, mag = X.product64(c.rows, c.off, c.w)
    if keep:
        c.check(pre, want, mag, K, "pre")
    assert (out[~c.inside] == POISON).all()
    h, off = gate64(want, mag * X.SUM(K))
    assert_close(out[c.inside], h[c.inside], X.bf16_tol(h, off)[c.inside], "out")


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,F,K,first,behind", GATES)
def test_gate_up_backward(ep, sizes, F, K, first, behind, kind):
    log(f"[bf16 gate up back] {sizes[:6]} F={F} K={K} {kind}")
    c = Case(sizes, 2 * F, K, first, behind, seed=2)
    pre, d = c.values(c.M, 2 * F), c.values(c.M, F)
    pre[~c.inside] = float("nan")
    d[~c.inside] = float("nan")
    grad_pre, grad_rows = torch.full((c.M, 2 * F), POISON, **BF), torch.full((c.M, K), POISON, **BF)
    grad_w = torch.full((c.G, 2 * F, K), POISON, dtype=kind, device="cuda")
    ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, pre, d, grad_pre, grad_rows, grad_w, c.st, c.workspace(ep))
    assert int(c.st) == 0
    p = pre[c.inside].double().requires_grad_(True)
    y = torch.nn.functional.silu(p[:, :F]) * p[:, F:]
    want, = torch.autograd.grad(y, p, d[c.inside].double())
    # the sigmoid (five roundings), 1 - s, the product-sum, three products; 1 + g (1 - s)
    # cancels at g = -1.28, where its parts are 1.28 each
    size = (d[c.inside].double() * torch.sigmoid(p[:, :F])).abs()
    g, u = p[:, :F].abs(), p[:, F:].abs()
    off = torch.cat([size * u * (2 + g), size * g], 1).detach() * 16 * X.U32
    assert (grad_pre[~c.inside] == POISON).all()
    assert_close(grad_pre[c.inside], want, X.bf16_tol(want, off), "grad_pre")
    # the products' gradients are those of the rounded one
    done = torch.where(c.inside[:, None], grad_pre, 0.0)
    c.check(grad_rows, *X.product64(done, c.off, c.w.transpose(1, 2)), 2 * F, "grad_rows")
    c.close(grad_w, *X.weights64(c.rows, c.off, done), max(sizes), "grad_w")
    # in pre's place, and without the products
    r, w = torch.full_like(grad_rows, POISON), torch.full_like(grad_w, POISON)
    inside = pre.clone()
    ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, inside, d, inside, r, w, c.st, c.workspace(ep, 0))
    assert torch.equal(inside[c.inside], grad_pre[c.inside]) and torch.isnan(inside[~c.inside]).all()
    assert torch.equal(r, grad_rows) and torch.equal(w, grad_w)
    again = torch.full_like(grad_pre, POISON)
    ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, pre, d, again, None, None, c.st)
    assert torch.equal(again, grad_pre) and int(c.st) == 0


# many rows an expert: tiles of one to several blocks, several tiles a workgroup, more
# experts than lanes, experts without rows among large ones
MANY = [([200], 8, 8), ([300], 264, 64), ([256], 256, 72), ([257, 255], 520, 128), ([513], 24, 136), ([150, 400], 512, 200),
        ([9000], 2056, 72), ([5000, 0, 4500], 1096, 8), ([130 + i % 7 for i in range(70)], 264, 136), ([0, 3000, 0, 0, 10, 2000], 520, 328),
        ([20000], 64, 64), ([140] * 40, 328, 1032)]


@pytest.mark.parametrize("sizes,N,K", MANY)
def test_many_rows(ep, sizes, N, K):
    log(f"[bf16 many rows] {sizes[:6]} N={N} K={K}")
    c = Case(sizes, N, K, 3, 5, whole=True, seed=11)
    out, gr = torch.full((c.M, N), POISON, **BF), torch.full((c.M, K), POISON, **BF)
    ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
    c.check(out, *X.product64(c.rows, c.off, c.w), K, "out")
    for kind in (torch.bfloat16, torch.float32):
        gw = torch.full((c.G, N, K), POISON, dtype=kind, device="cuda")
        gr.fill_(POISON)
        ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, c.workspace(ep))
        c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), N, "grad_rows")
        c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), max(sizes), "grad_w")
    F = N // 2
    if F % 8 == 0:
        pre, h = torch.full((c.M, N), POISON, **BF), torch.full((c.M, F), POISON, **BF)
        ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre, h, c.st)
        want, mag = X.product64(c.rows, c.off, c.w)
        c.check(pre, want, mag, K, "pre")
        assert (h[~c.inside] == POISON).all()
        act, off = gate64(want, torch.zeros_like(want))
        assert_close(h[c.inside], act[c.inside], X.bf16_tol(act, off)[c.inside], "gated")
    assert int(c.st) == 0


def test_gates_far_from_zero(ep):
    """One row, one weight: the gates are what they are said to be."""
    g = [-3e38, -1e4, -205.0, -199.0, -103.5, -95.0, -89.0, -88.5, -87.0, -80.5, -79.5, -20.0, -1.0, -1e-30, 0.0, 1e-30, 1.0, 20.0, 88.0, 3e38,
         float("inf"), float("-inf"), float("nan"), 0.5]
    F, K = len(g), 8
    w = torch.zeros(1, 2 * F, K, **BF)
    w[0, :F, 0] = torch.tensor(g)
    w[0, F:, 0] = 3.0
    rows = torch.zeros(1, K, **BF)
    rows[0, 0] = 1.0
    off, st = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, F, **BF)
    for copies in (1, 300):        # small and big tiles
        x = rows.repeat(copies, 1)
        out = torch.zeros(copies, F, **BF)
        off[1] = copies
        ep.ep_expert_gate_up_bf16(x, off, w, None, out, st)
        gate = w[0, :F, 0].double()
        want = torch.where(gate == float("-inf"), float("nan"), gate * torch.sigmoid(gate) * 3.0).expand(copies, F)
        want = torch.where(want.abs() > 3.4e38, want.bfloat16().double(), want)      # beyond bf16: infinite
        tol = X.bf16_tol(want, 8 * 4 * X.U32 * want.abs() + (gate * 3.0).abs() * 2.0 ** -149)
        assert_close(out, want, torch.nan_to_num(tol, 0.0, 0.0, 0.0), "gated")


def test_a_long_sum_in_parts(ep):
    """Few weights, many rows: the weights' gradient is summed in parts."""
    for sizes, N, K in (([30000], 64, 72), ([5000, 0, 9000], 264, 520), ([700], 8, 8)):
        c = Case(sizes, N, K, 1, 2, whole=True, seed=12)
        assert sum(sizes) < 1000 or ep.ep_expert_backward_workspace_bytes(c.G, c.M, N, K) > 0
        for kind in (torch.bfloat16, torch.float32):
            gw = torch.full((c.G, N, K), POISON, dtype=kind, device="cuda")
            ep.ep_expert_product_bf16_backward(c.rows, c.off, None, c.grad_out, None, gw, c.st, c.workspace(ep))
            c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), max(sizes), "grad_w")
        assert int(c.st) == 0


def test_differences(ep):
    """Central differences of the library's own forward in a direction, against its
    gradients: whole numbers make the plain product exact."""
    c = Case([40, 0, 25], 72, 136, whole=True, seed=5)
    grad_rows, grad_w = torch.zeros(c.M, 136, **BF), torch.zeros(3, 72, 136, device="cuda")
    ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, grad_rows, grad_w, c.st, c.workspace(ep))
    exact, _ = X.product64(c.grad_out, c.off, c.w.transpose(1, 2))
    f = lambda rows, w: X.product64(rows, c.off, w)[0]  # noqa: E731
    step_r, step_w = c.values(c.M, 136), c.values(3, 72, 136)
    d = c.grad_out.double()
    by_rows = (d * (f(c.rows + step_r, c.w) - f(c.rows - step_r, c.w))).sum() / 2
    by_w = (d * (f(c.rows, c.w + step_w) - f(c.rows, c.w - step_w))).sum() / 2
    assert by_rows == (exact * step_r.double()).sum() and torch.equal(grad_rows, exact.bfloat16())
    assert by_w == (grad_w.double() * step_w.double()).sum()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_infinite_and_nan_values_stay_in_their_rows_and_experts(ep, bad):
    c = Case([70, 3, 90], 136, 200, whole=True, seed=6)
    clean = Case([70, 3, 90], 136, 200, whole=True, seed=6)
    row, e = 75, 1                                     # a row of expert 2; a weight of expert 1
    c.rows[row, 33] = bad
    c.w[e, 100, 199] = bad
    out, want = torch.zeros(c.M, 136, **BF), torch.zeros(c.M, 136, **BF)
    ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
    ep.ep_expert_product_bf16(clean.rows, c.off, clean.w, want, c.st)
    other = torch.ones(c.M, 136, dtype=torch.bool, device="cuda")
    other[row] = False
    other[70:73, 100] = False
    assert torch.equal(out[other], want[other])
    assert not torch.isfinite(out[row]).any()
    c = Case([70, 3, 90], 136, 200, whole=True, seed=6)
    c.grad_out[row, 50] = bad
    c.w[e, 100, 199] = bad
    got, want = [], []
    for d, to in ((c, got), (clean, want)):
        to += [torch.zeros(c.M, 200, **BF), torch.zeros(3, 136, 200, **BF)]
        ep.ep_expert_product_bf16_backward(c.rows, c.off, d.w, d.grad_out, to[0], to[1], c.st, c.workspace(ep))
    other = torch.ones(c.M, 200, dtype=torch.bool, device="cuda")
    other[row] = False
    other[70:73, 199] = False
    assert torch.equal(got[0][other], want[0][other])
    other = torch.ones(3, 136, 200, dtype=torch.bool, device="cuda")
    other[2, 50] = False
    assert torch.equal(got[1][other], want[1][other])
    assert not torch.isfinite(got[1][2, 50][c.rows[row] != 0]).any()


def test_offsets_that_do_not_fit(ep):
    N, K, M = 72, 80, 100
    g = torch.Generator(device="cuda").manual_seed(0)
    rows, w = torch.randn(M, K, device="cuda", generator=g).bfloat16(), torch.randn(3, N, K, device="cuda", generator=g).bfloat16()
    d = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    for off, code in (([0, 10, 20, 101], ep.EP_ERR_CAPACITY), ([0, 30, 20, 100], ep.EP_ERR_INVALID_ARG),
                      ([-5, 10, 20, 100], ep.EP_ERR_INVALID_ARG), ([0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], ep.EP_ERR_CAPACITY)):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        big = torch.full((3 * M, N), POISON, **BF)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.ep_expert_product_bf16(rows, o, w, big[M:2 * M], st)
        assert int(st) == code
        assert (big[:M] == POISON).all() and (big[2 * M:] == POISON).all()
        st.zero_()
        back, gw = torch.full((3 * M, K), POISON, **BF), torch.full((5, N, K), POISON, **BF)
        ep.ep_expert_product_bf16_backward(rows, o, w, d, back[M:2 * M], gw[1:4], st,
                                           torch.empty(ep.ep_expert_backward_workspace_bytes(3, M, N, K) + 16, dtype=torch.uint8, device="cuda"))
        assert int(st) == code
        assert (back[:M] == POISON).all() and (back[2 * M:] == POISON).all() and (gw[0] == POISON).all() and (gw[4] == POISON).all()


def test_no_rows(ep):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w, st = torch.ones(3, 64, 72, **BF), torch.zeros(1, dtype=torch.int32, device="cuda")
    e = lambda n: torch.empty(0, n, **BF)  # noqa: E731
    ep.ep_expert_product_bf16(e(72), off, w, e(64), st)
    ep.ep_expert_gate_up_bf16(e(72), off, w, e(64), e(32), st)
    for kind in (torch.bfloat16, torch.float32):
        gw = torch.full((3, 64, 72), POISON, dtype=kind, device="cuda")
        ep.ep_expert_product_bf16_backward(e(72), off, w, e(64), e(72), gw, st)
        assert (gw == 0).all()
        gw.fill_(POISON)
        ep.ep_expert_gate_up_bf16_backward(e(72), off, w, e(64), e(32), e(64), e(72), gw, st)
        assert (gw == 0).all() and int(st) == 0


def test_many_experts(ep):
    """More experts than a wavefront has lanes, most without rows."""
    sizes = [(i * 7) % 5 * (i % 3 == 0) for i in range(600)]
    c = Case(sizes, 24, 40, 3, 3, whole=True)
    out, gr = torch.full((c.M, 24), POISON, **BF), torch.full((c.M, 40), POISON, **BF)
    gw = torch.full((600, 24, 40), POISON, device="cuda")
    ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
    ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, c.workspace(ep))
    c.check(out, *X.product64(c.rows, c.off, c.w), 40, "out")
    c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), 24, "grad_rows")
    c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), 4, "grad_w")
    assert int(c.st) == 0


def test_captured(ep):
    """A forward and a backward in one graph, replayed on other inputs and offsets
    with the program's own work between."""
    F, K, M = 72, 136, 300
    c = Case([100, 50, 150], 2 * F, K, seed=7)
    pre, inner = torch.zeros(M, 2 * F, **BF), torch.zeros(M, F, **BF)
    gp, gr, gw = torch.zeros(M, 2 * F, **BF), torch.zeros(M, K, **BF), torch.zeros(3, 2 * F, K, device="cuda")
    d, ws = c.values(M, F), c.workspace(ep)

    def step():
        ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre, inner, c.st)
        ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, pre, d, gp, gr, gw, c.st, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, off in enumerate(([0, 100, 150, 300], [0, 0, 299, 300], [0, 1, 2, 3], [10, 10, 10, 200])):
        c.off.copy_(torch.tensor(off, dtype=torch.int32))
        c.rows.copy_(c.values(M, K))
        outs = (pre, inner, gp, gr, gw)
        for t in outs:
            t.fill_(POISON)
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(POISON)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
    assert int(c.st) == 0


def test_two_streams(ep):
    """Two calls at once, on streams of their own, each with its workspace."""
    a, b = Case([900, 100], 264, 328, whole=True, seed=8), Case([50, 950], 264, 328, whole=True, seed=9)
    side, got = torch.cuda.Stream(), []
    bufs = [(torch.full((c.M, 328), POISON, **BF), torch.full((2, 264, 328), POISON, device="cuda"), c.workspace(ep)) for c in (a, b)]
    side.wait_stream(torch.cuda.current_stream())
    for c, (gr, gw, ws), s in ((a, bufs[0], None), (b, bufs[1], side)):
        for _ in range(3):
            ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, ws, s)
    torch.cuda.synchronize()
    for c, (gr, gw, _) in zip((a, b), bufs):
        c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), 264, "grad_rows")
        c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), 950, "grad_w")


def test_refusals(ep):
    c = Case([4, 5], 64, 72)
    out, gr, gw = torch.zeros(9, 64, **BF), torch.zeros(9, 72, **BF), torch.zeros(2, 64, 72, **BF)
    good = dict(rows=c.rows, group_offset=c.off, w=c.w, out=out, dev_status=c.st)
    bad = [dict(rows=None), dict(rows=c.rows.float()), dict(rows=c.rows[:, :64]), dict(rows=c.rows.t()), dict(group_offset=c.off[:2]),
           dict(group_offset=c.off.long()), dict(w=None), dict(w=c.w[0]), dict(w=c.w.half()), dict(w=c.w.transpose(1, 2)),
           dict(out=None), dict(out=out[:8]), dict(out=out.float()), dict(dev_status=None), dict(rows=c.rows.cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            ep.ep_expert_product_bf16(**{**good, **b})
    good = dict(rows=c.rows, group_offset=c.off, w=c.w, grad_out=c.grad_out, grad_rows=gr, grad_w=gw, dev_status=c.st)
    bad = [dict(grad_rows=None, grad_w=None), dict(rows=None), dict(w=None), dict(grad_out=None), dict(grad_out=c.grad_out[:, :32]),
           dict(grad_w=gw.half()), dict(grad_w=gw[:1]), dict(grad_rows=gr[:, :64]), dict(grad_rows=gr.float())]
    for b in bad:
        with pytest.raises(ValueError):
            ep.ep_expert_product_bf16_backward(**{**good, **b})
    big = Case([4000], 64, 72)
    with pytest.raises(ValueError):      # this one needs a workspace
        ep.ep_expert_product_bf16_backward(big.rows, big.off, big.w, big.grad_out, None, torch.zeros(1, 64, 72, **BF), big.st)
    with pytest.raises(ep.EpError):
        ep.ep_expert_product_bf16_backward(big.rows, big.off, big.w, big.grad_out, None, torch.zeros(1, 64, 72, **BF), big.st,
                                           torch.zeros(64, dtype=torch.uint8, device="cuda"))
    odd = Case([4], 24, 72)
    with pytest.raises(ep.EpError):      # F = 12
        ep.ep_expert_gate_up_bf16(odd.rows, odd.off, odd.w, None, torch.zeros(4, 12, **BF), odd.st)
    odd = Case([4], 12, 72)
    with pytest.raises(ep.EpError):
        ep.ep_expert_product_bf16(odd.rows, odd.off, odd.w, torch.zeros(4, 12, **BF), odd.st)


def test_rows_without_two_dimensions(ep):
    c = Case([4, 5], 64, 72)
    out, gw = torch.zeros(9, 64, **BF), torch.zeros(2, 64, 72, **BF)
    for rows in (c.rows[0], c.rows[0, 0], c.rows[None]):
        with pytest.raises(ValueError):
            ep.ep_expert_product_bf16(rows, c.off, c.w, out, c.st)
        with pytest.raises(ValueError):
            ep.ep_expert_product_bf16_backward(rows, c.off, None, c.grad_out, None, gw, c.st)
    with pytest.raises(ValueError):
        ep.ep_expert_product_bf16_backward(None, c.off, c.w, c.grad_out[0, 0], torch.zeros(9, 72, **BF), None, c.st)
