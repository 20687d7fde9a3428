"""The big tiles of the bf16 expert products: every case here is one that the rule
sends to them, which ep_expert_bf16_plan says and each test asserts, so that a rule
that changes cannot leave them untested.

Inputs and tolerances are those of test_gpu_expert_bf16.py: small whole numbers, whose
result is bit for bit the rounded 64-bit one, and random ones."""

import pytest
import torch

import training_refs as X
from gpu_helpers import log
from operator_refs import assert_close
from test_gpu_expert_bf16 import BF, POISON, Case, gate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def needs_big(ep, c, products):
    """Whether the products (F forward, G gate and up, R the rows' gradient, W the weights') take big tiles."""
    for p in products:
        assert ep.ep_expert_bf16_plan("FGRW".index(p), c.G, c.M, c.N, c.K) == ep.EP_TILES_BIG, (p, c.G, c.M, c.N, c.K)


# sizes of the groups, N, K, which products take big tiles
CASES = [
    # columns, rows and c that end inside a tile or a block; an expert without rows
    ([3000, 0, 3001], 1096, 1032, "FRW"),
    ([513, 1, 255, 0, 2000, 700], 2064, 2056, "FGRW"),
    # several tiles a workgroup, one column tile that is nearly empty
    ([5900, 100], 2064, 264, "FW"),
    ([20000], 2064, 264, "FGRW"),
    # more experts than a wavefront has lanes; every second one without rows
    ([100] * 70, 2064, 1032, "FGRW"),
    ([300, 0] * 70, 1040, 520, "FGRW"),
    # one block of c, whole and not; two, the second not whole: tiles that begin and end in a block
    ([30000, 100], 1552, 64, "FW"),
    ([60000], 1040, 48, "FW"),
    ([40000, 0, 3000], 1552, 72, "FW"),
    ([26000, 0, 34000], 2032, 56, "G"),
    ([40000, 100, 25000], 2032, 72, "G"),
    ([30000, 100], 64, 1552, "RW"),
    ([16000], 56, 2072, "RW"),
    ([20000], 72, 2064, "RW"),
]


@pytest.mark.parametrize("sizes,N,K,products", CASES)
def test_whole_numbers(ep, sizes, N, K, products):
    log(f"[bf16 big tiles] {len(sizes)} {sizes[:6]} N={N} K={K} {products}")
    c = Case(sizes, N, K, 3, 5, whole=True, seed=21)
    needs_big(ep, c, products)
    if "F" in products:
        out = torch.full((c.M, N), POISON, **BF)
        ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
        c.check(out, *X.product64(c.rows, c.off, c.w), K, "out")
    if "G" in products:
        want, mag = X.product64(c.rows, c.off, c.w)
        act, off = gate64(want, torch.zeros_like(want))
        for keep in (True, False):
            pre, h = torch.full((c.M, N), POISON, **BF), torch.full((c.M, N // 2), POISON, **BF)
            ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre if keep else None, h, c.st)
            if keep:
                c.check(pre, want, mag, K, "pre")
            assert (h[~c.inside] == POISON).all()
            assert_close(h[c.inside], act[c.inside], X.bf16_tol(act, off)[c.inside], "gated")
    if "R" in products:
        gr = torch.full((c.M, K), POISON, **BF)
        ep.ep_expert_product_bf16_backward(None, c.off, c.w, c.grad_out, gr, None, c.st)
        c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), N, "grad_rows")
    if "W" in products:
        want = X.weights64(c.rows, c.off, c.grad_out)
        for kind in (torch.bfloat16, torch.float32):
            gw = torch.full((c.G, N, K), POISON, dtype=kind, device="cuda")
            ep.ep_expert_product_bf16_backward(c.rows, c.off, None, c.grad_out, None, gw, c.st, c.workspace(ep))
            c.close(gw, *want, max(sizes), "grad_w")
    assert int(c.st) == 0


@pytest.mark.parametrize("sizes,N,K", [([513, 1, 255, 0, 2000, 700], 2064, 2056), ([100] * 70, 2064, 1032), ([20000], 2064, 264)])
def test_random_numbers(ep, sizes, N, K):
    """Forward, gate and both backward calls, on random numbers."""
    log(f"[bf16 big tiles] random {len(sizes)} {sizes[:6]} N={N} K={K}")
    c = Case(sizes, N, K, 2, 1, seed=22)
    needs_big(ep, c, "FGRW")
    c.w *= K ** -0.5
    F = N // 2
    out, pre, h = torch.full((c.M, N), POISON, **BF), torch.full((c.M, N), POISON, **BF), torch.full((c.M, F), POISON, **BF)
    ep.ep_expert_product_bf16(c.rows, c.off, c.w, out, c.st)
    ep.ep_expert_gate_up_bf16(c.rows, c.off, c.w, pre, h, c.st)
    want, mag = X.product64(c.rows, c.off, c.w)
    c.check(out, want, mag, K, "out")
    c.check(pre, want, mag, K, "pre")
    assert (h[~c.inside] == POISON).all()
    act, off = gate64(want, mag * X.SUM(K))
    assert_close(h[c.inside], act[c.inside], X.bf16_tol(act, off)[c.inside], "gated")
    for kind in (torch.bfloat16, torch.float32):
        gr, gp = torch.full((c.M, K), POISON, **BF), torch.full((c.M, N), POISON, **BF)
        gw = torch.full((c.G, N, K), POISON, dtype=kind, device="cuda")
        ep.ep_expert_product_bf16_backward(c.rows, c.off, c.w, c.grad_out, gr, gw, c.st, c.workspace(ep))
        c.check(gr, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), N, "grad_rows")
        c.close(gw, *X.weights64(c.rows, c.off, c.grad_out), max(sizes), "grad_w")
        d = c.grad_out[:, :F].contiguous()
        ep.ep_expert_gate_up_bf16_backward(c.rows, c.off, c.w, pre, d, gp, gr, gw, c.st, c.workspace(ep))
        done = torch.where(c.inside[:, None], gp, 0.0)
        c.check(gr, *X.product64(done, c.off, c.w.transpose(1, 2)), N, "grad_rows of the gate's")
        c.close(gw, *X.weights64(c.rows, c.off, done), max(sizes), "grad_w of the gate's")
    assert int(c.st) == 0


def test_gates_far_from_zero(ep):
    """One column of rows and weights: the gates are what they are said to be."""
    g = [-3e38, -1e4, -205.0, -199.0, -103.5, -95.0, -89.0, -88.5, -87.0, -80.5, -79.5, -20.0, -1.0, -1e-30, 0.0, 1e-30, 1.0, 20.0, 88.0, 3e38,
         float("inf"), float("-inf"), float("nan"), 0.5] * 43
    F, K, M = len(g), 264, 20000
    assert ep.ep_expert_bf16_plan(ep.EP_PRODUCT_GATE_UP, 1, M, 2 * F, K) == ep.EP_TILES_BIG
    w = torch.zeros(1, 2 * F, K, **BF)
    w[0, :F, 0] = torch.tensor(g)
    w[0, F:, 0] = 3.0
    rows = torch.zeros(M, K, **BF)
    rows[:, 0] = 1.0
    off, st = torch.tensor([0, M], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(M, F, **BF)
    ep.ep_expert_gate_up_bf16(rows, off, w, None, out, st)
    assert int(st) == 0
    gate = w[0, :F, 0].double()
    want = torch.where(gate == float("-inf"), float("nan"), gate * torch.sigmoid(gate) * 3.0)
    want = torch.where(want.abs() > 3.4e38, want.bfloat16().double(), want)      # beyond bf16: infinite
    tol = X.bf16_tol(want, 8 * 4 * X.U32 * want.abs() + (gate * 3.0).abs() * 2.0 ** -149)
    assert_close(out, want.expand(M, F), torch.nan_to_num(tol, 0.0, 0.0, 0.0).expand(M, F), "gated")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_infinite_and_nan_values_stay_in_their_rows_and_experts(ep, bad):
    sizes, N, K = [700, 3, 2300, 600], 2064, 2056
    clean = Case(sizes, N, K, whole=True, seed=23)
    needs_big(ep, clean, "FGRW")
    row, e = 2500, 1                          # a row of expert 2; weights of expert 1
    c = Case(sizes, N, K, whole=True, seed=23)
    c.rows[row, 33] = bad
    c.w[e, 100, K - 1] = bad
    got, want = [], []
    for d, to in ((c, got), (clean, want)):
        to += [torch.zeros(c.M, N, **BF), torch.zeros(c.M, N, **BF), torch.zeros(c.M, N // 2, **BF)]
        ep.ep_expert_product_bf16(d.rows, c.off, d.w, to[0], c.st)
        ep.ep_expert_gate_up_bf16(d.rows, c.off, d.w, to[1], to[2], c.st)
    other = torch.ones(c.M, N, dtype=torch.bool, device="cuda")
    other[row] = False
    other[700:703, 100] = False
    assert torch.equal(got[0][other], want[0][other]) and torch.equal(got[1][other], want[1][other])
    assert not torch.isfinite(got[0][row][c.w[2, :, 33] != 0]).any()
    other = other[:, :N // 2]                # column 100 is a gate's
    assert torch.equal(got[2][other], want[2][other])
    c = Case(sizes, N, K, whole=True, seed=23)
    c.grad_out[row, 50] = bad
    c.w[e, 100, K - 1] = bad
    got, want = [], []
    for d, to in ((c, got), (clean, want)):
        to += [torch.zeros(c.M, K, **BF), torch.zeros(4, N, K, **BF)]
        ep.ep_expert_product_bf16_backward(c.rows, c.off, d.w, d.grad_out, to[0], to[1], c.st, c.workspace(ep))
    other = torch.ones(c.M, K, dtype=torch.bool, device="cuda")
    other[row] = False
    other[700:703, K - 1] = False
    assert torch.equal(got[0][other], want[0][other])
    other = torch.ones(4, N, K, dtype=torch.bool, device="cuda")
    other[2, 50] = False
    assert torch.equal(got[1][other], want[1][other])
    assert not torch.isfinite(got[1][2, 50][c.rows[row] != 0]).any()
    assert int(c.st) == 0


def test_offsets_that_do_not_fit(ep):
    """Offsets behind M, below zero or falling: reported, and no row beside the buffers' is written."""
    c = Case([3000, 0, 3001], 1096, 1032, seed=24)
    needs_big(ep, c, "FRW")
    M = c.M
    for off, code in (([0, 3000, 3000, M + 1], ep.EP_ERR_CAPACITY), ([0, 4000, 2000, M], ep.EP_ERR_INVALID_ARG),
                      ([-5, 10, 20, M], ep.EP_ERR_INVALID_ARG), ([0, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], ep.EP_ERR_CAPACITY)):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        out, back = torch.full((M + 600, c.N), POISON, **BF), torch.full((M + 600, c.K), POISON, **BF)
        gw = torch.full((5, c.N, c.K), POISON, **BF)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ep.ep_expert_product_bf16(c.rows, o, c.w, out[300:300 + M], st)
        assert int(st) == code
        st.zero_()
        ep.ep_expert_product_bf16_backward(c.rows, o, c.w, c.grad_out, back[300:300 + M], gw[1:4], st, c.workspace(ep))
        assert int(st) == code
        for t in (out, back):
            assert (t[:300] == POISON).all() and (t[300 + M:] == POISON).all()
        assert (gw[0] == POISON).all() and (gw[4] == POISON).all()


@pytest.mark.parametrize("rows_at,w_at", [(0, 1), (3, 0), (7, 5)])
def test_operands_off_lines(ep, rows_at, w_at):
    """Tensors that begin 16 bytes times rows_at and w_at behind a line, NaN around them."""
    c = Case([3000, 0, 3001], 1096, 1032, whole=True, seed=25)
    needs_big(ep, c, "FRW")

    def moved(x, at):
        room = torch.full((x.numel() + 192,), float("nan"), **BF)
        room = room[-room.data_ptr() % 128 // 2:]
        y = room[8 * at:][:x.numel()].view(x.shape)
        assert y.data_ptr() % 128 == 16 * at
        return y.copy_(x)

    rows, w, grad_out = moved(c.rows, rows_at), moved(c.w, w_at), moved(c.grad_out, w_at)
    out, grad_rows = torch.full((c.M, c.N), POISON, **BF), torch.full((c.M, c.K), POISON, **BF)
    grad_w = torch.full_like(w, POISON)
    ep.ep_expert_product_bf16(rows, c.off, w, out, c.st)
    ep.ep_expert_product_bf16_backward(rows, c.off, w, grad_out, grad_rows, grad_w, c.st, c.workspace(ep))
    assert int(c.st) == 0
    c.check(out, *X.product64(c.rows, c.off, c.w), c.K, "out")
    c.check(grad_rows, *X.product64(c.grad_out, c.off, c.w.transpose(1, 2)), c.N, "grad_rows")
    c.close(grad_w, *X.weights64(c.rows, c.off, c.grad_out), 3001, "grad_w")
