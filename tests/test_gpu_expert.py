"""ep_expert_product and ep_expert_gate_up against 64 bits.

Exact cases: codes of small whole numbers and scales that are powers of two make
every product and sum exact in float, whatever the order, so the product equals
the 64-bit one rounded once, bit for bit.  Random cases: operator_refs.mfma_bound
and the output's rounding."""

import numpy as np
import pytest
import torch

import operator_refs as R
from gpu_helpers import log

pytestmark = pytest.mark.gpu

# counts of each group's rows, N (or F), K
PRODUCT = [([1], 8, 128), ([1], 16, 256), ([3], 24, 384), ([16], 128, 128), ([17], 136, 512), ([0, 5, 0, 1], 64, 128),
           ([2, 0, 31, 7], 264, 640), ([1] * 70, 40, 128), ([0] * 65 + [4], 72, 256), ([33, 64, 65], 200, 384),
           ([128, 127, 129, 0, 1], 512, 512), ([300], 1000, 896), ([255, 257, 0, 513], 520, 1792),
           ([40, 1000, 3], 1208, 256), ([700], 256, 128), ([300], 8, 128),
           ([20, 19, 64, 1], 40, 384), ([530], 304, 640), ([9] * 40, 264, 256), ([8] * 33 + [250], 376, 512)]
GATE_UP = [([1], 128, 128), ([3], 128, 256), ([16, 17], 256, 384), ([0, 5, 0, 1], 384, 128), ([2, 0, 31, 7], 128, 640),
           ([1] * 70, 128, 128), ([33, 64, 65], 256, 384), ([128, 127, 129, 0, 1], 640, 512), ([300], 896, 896),
           ([255, 257, 0, 513], 128, 1792), ([40, 1000, 3], 384, 256), ([16] * 5, 128, 2304),
           ([15, 17, 1], 256, 2176), ([11], 128, 4096), ([600], 128, 128), ([17] * 40, 256, 256)]


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def offsets(counts, first=0):
    return [first + int(v) for v in np.concatenate([[0], np.cumsum(counts)])]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def exact_inputs(M, G, N, K, gen):
    """Codes of -2 .. 2 and scales of powers of two, and their values."""
    def codes(*shape):
        v = torch.randint(-2, 3, shape, device="cuda", generator=gen).float()
        return v.to(torch.float8_e4m3fn)

    def scales(*shape):
        return torch.exp2(torch.randint(-3, 4, shape, device="cuda", generator=gen).float())

    x, sx = codes(M, K), scales(M, K // 128)
    rows = torch.full((M, R.row_bytes(K)), 0x5A, dtype=torch.uint8, device="cuda")   # the pad is not read
    rows[:, :K] = x.view(torch.uint8)
    rows[:, K:K + K // 32] = sx.view(torch.uint8)
    w, sw = codes(G, N, K), scales(G, -(-N // 128), K // 128)
    return (rows, x.double() * sx.double().repeat_interleave(128, 1), w.view(torch.uint8), sw, R.weights64(w, sw))


def product(ep, rows, off, w, sw, M, N, stream=None):
    out = torch.full((M, N), -7.0, dtype=torch.bfloat16, device="cuda")
    st = i32([0])
    ep.ep_expert_product(rows, i32(off), w, sw, out, st, stream=stream)
    return out, int(st)


def gate_up(ep, rows, off, w, sw, M, F):
    out = torch.full((M, R.row_bytes(F)), 0xA5, dtype=torch.uint8, device="cuda")
    st = i32([0])
    ep.ep_expert_gate_up(rows, i32(off), w, sw, out, st)
    return out, int(st)


@pytest.mark.parametrize("counts,N,K", PRODUCT)
@pytest.mark.parametrize("first,behind", [(0, 0), (5, 9)])
def test_product_exact(ep, counts, N, K, first, behind):
    gen = torch.Generator(device="cuda").manual_seed(1)
    off = offsets(counts, first)
    M, G = off[-1] + behind, len(counts)
    rows, x, w, sw, w64 = exact_inputs(M, G, N, K, gen)
    log(f"[product] counts={counts[:6]} N={N} K={K}")
    out, st = product(ep, rows, off, w, sw, M, N)
    assert st == 0
    want = R.grouped64(x, off, w64)
    inside = slice(first, off[-1])
    assert torch.equal(out[inside], want[inside].float().bfloat16())
    assert (out[:first] == -7).all() and (out[off[-1]:] == -7).all()


@pytest.mark.parametrize("counts,N,K", [([7, 0, 1, 20], 392, 7168), ([128, 300, 50], 712, 1792), ([600], 640, 7168)])
def test_product_random(ep, counts, N, K):
    gen = torch.Generator(device="cuda").manual_seed(2)
    off = offsets(counts)
    M, G = off[-1], len(counts)
    rows, x = R.make_rows(torch.randn(M, K, device="cuda", generator=gen) * 3)
    w, sw, w64 = R.make_weights(G, N, K, gen)
    out, st = product(ep, rows, off, w, sw, M, N)
    assert st == 0
    want = R.grouped64(x, off, w64)
    R.assert_close(out, want, want.abs() * R.U_BF16 + R.mfma_bound(x, off, w64), "out")
    # over all outputs: bf16's rounding, and what the matrix unit drops, at
    # most 2^-13 of each eight's largest product in either direction
    assert float((out.double() - want).norm() / want.norm()) <= R.U_BF16 + 2.0 ** -13


@pytest.mark.parametrize("counts,F,K", GATE_UP)
@pytest.mark.parametrize("first,behind", [(0, 0), (3, 6)])
def test_gate_up_exact(ep, counts, F, K, first, behind):
    """The two products are exact; silu(gate) * up is off by exp's rounding of
    its argument, two of its own, the quotient's and the product's."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    off = offsets(counts, first)
    M, G = off[-1] + behind, len(counts)
    rows, x, w, sw, _ = exact_inputs(M, G, 2 * F, K, gen)
    sw = sw * 2.0 ** -6          # gates where silu bends
    w64 = R.weights64(w.view(torch.float8_e4m3fn), sw)
    log(f"[gate_up] counts={counts[:6]} F={F} K={K}")
    out, st = gate_up(ep, rows, off, w, sw, M, F)
    assert st == 0
    y = R.grouped64(x, off, w64)[first:off[-1]]
    g, u = y[:, :F], y[:, F:]
    h = g / (1 + torch.exp(-g)) * u
    big = g.abs().view(g.shape[0], -1, 128).amax(2)
    R.assert_rows8(out[first:off[-1]], h, (big + 6) * R.U32, "out_rows")
    assert (out[:first] == 0xA5).all() and (out[off[-1]:] == 0xA5).all()


def test_gate_up_random(ep):
    """Against 64 bits from the same 8-bit inputs: gate and up are each off by
    2^-13 of their norm at most, h by twice that; a code then by half a step."""
    counts, F, K = [30, 0, 200, 1], 512, 7168
    gen = torch.Generator(device="cuda").manual_seed(4)
    off = offsets(counts)
    M = off[-1]
    rows, x = R.make_rows(torch.randn(M, K, device="cuda", generator=gen))
    w, sw, w64 = R.make_weights(len(counts), 2 * F, K, gen)
    out, st = gate_up(ep, rows, off, w, sw, M, F)
    y = R.grouped64(x, off, w64)
    h = torch.nn.functional.silu(y[:, :F]) * y[:, F:]
    codes, scales, pad = R.split_rows(out, F)
    assert st == 0 and not pad.any()
    got = codes * scales.repeat_interleave(128, 1)
    a = h.abs().view(M, -1, 128).amax(2).repeat_interleave(128, 1)
    # 2^-9 of the block's largest: gates and ups of size 1 that the unit moved
    # by less than that, on top of the code's half step
    R.assert_close(got, h, h.abs() * R.U_E4M3 * 1.01 + a * 2.0 ** -9, "h")
    assert float((got - h).norm() / h.norm()) <= R.U_E4M3


def test_large_gates_do_not_overflow(ep):
    """silu far out: exp overflows to infinity for gates below -89 (h = -0) and
    vanishes above (h = gate * up); infinite and NaN inputs stay in their row."""
    K, F = 128, 128
    rows = torch.zeros(4, R.row_bytes(K), dtype=torch.uint8, device="cuda")
    one = torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8).item()
    rows[:, 0] = one
    rows[:, K:K + 4] = torch.ones(4, 1, device="cuda").view(torch.uint8)
    rows[2, 1] = 0x7F                                        # a NaN code
    rows[3, K:K + 4] = torch.full((1,), float("inf"), device="cuda").view(torch.uint8)
    w = torch.zeros(1, 2 * F, K, device="cuda")
    w[0, :F, 0] = torch.linspace(-448, 448, F, device="cuda")
    w[0, F:, 0] = 2.0
    codes = w.to(torch.float8_e4m3fn)
    sw = torch.ones(1, 2, 1, device="cuda")
    out, st = gate_up(ep, rows, [0, 4], codes.view(torch.uint8), sw, 4, F)
    assert st == 0
    g = codes.double()[0, :F, 0]
    h = (g * torch.sigmoid(g) * 2.0)[None].repeat(2, 1)
    R.assert_rows8(out[:2], h, (g.abs().max() + 6).item() * R.U32, "rows")
    bad, _, _ = R.split_rows(out[2:], F)
    assert torch.isnan(bad[0]).all()          # NaN gates and ups
    assert torch.isnan(bad[1]).any()          # inf * 0 among the products


@pytest.mark.parametrize("which", ["product", "gate_up"])
def test_nan_rows_and_weights_stay_in_their_places(ep, which):
    gen = torch.Generator(device="cuda").manual_seed(5)
    counts, N, K = [20, 70, 3], 256, 256
    off = offsets(counts)
    M = off[-1]
    rows, x, w, sw, w64 = exact_inputs(M, 3, N, K, gen)
    f = product if which == "product" else gate_up
    n = N if which == "product" else N // 2
    clean, _ = f(ep, rows, off, w, sw, M, n)
    rows2 = rows.clone()
    rows2[25, 130] = 0x7F
    dirty, _ = f(ep, rows2, off, w, sw, M, n)
    same = [m for m in range(M) if m != 25]
    assert torch.equal(clean[same].view(torch.uint8), dirty[same].view(torch.uint8))
    assert not torch.equal(clean[25].view(torch.uint8), dirty[25].view(torch.uint8))
    if which == "product":
        assert torch.isnan(dirty[25]).all()
        w2 = w.clone()
        w2[1, 100, 7] = 0xFF
        dirty, _ = f(ep, rows, off, w2, sw, M, n)
        assert torch.isnan(dirty[20:90, 100]).all()
        ok = torch.ones_like(clean, dtype=torch.bool)
        ok[20:90, 100] = False
        assert torch.equal(clean[ok], dirty[ok])


def test_bad_offsets_are_reported(ep):
    gen = torch.Generator(device="cuda").manual_seed(6)
    M, N, K = 50, 128, 128
    rows, x, w, sw, w64 = exact_inputs(M, 3, N, K, gen)
    guard = torch.full((3 * M, N), -7.0, dtype=torch.bfloat16, device="cuda")
    for off, want in [([0, 10, 20, 51], 3), ([0, 30, 20, 50], 1), ([-1, 10, 20, 30], 1),
                      ([0, 10, 2 ** 31 - 1, 2 ** 31 - 1], 3), ([50, 0, 50, 0], 1)]:
        st = i32([0])
        out = guard[M:2 * M]
        ep.ep_expert_product(rows, i32(off), w, sw, out, st)
        assert int(st) == want
        assert (guard[:M] == -7).all() and (guard[2 * M:] == -7).all()
    # rows beyond M are skipped, the others computed
    out, st = product(ep, rows, [0, 10, 20, 51], w, sw, M, N)
    assert st == 3
    assert torch.equal(out[:20], R.grouped64(x, [0, 10, 20, 50], w64)[:20].float().bfloat16())


MIXED = [0, 64, 65, 1, 63, 128, 17, 0, 200, 3]
# Sizes that the middle and the big tiles take: middle ones for 9 to 48 rows a
# group or few tiles, big ones for more rows and more than 384 (gate: 352) middle
# tiles.
LARGER_PRODUCT = [([30] * 20, 1304, 512), (MIXED, 2056, 640), ([9] * 30, 8200, 128), ([40, 1, 0, 7] * 6, 4104, 256),
                  ([17, 33, 0, 66, 5] * 5, 2600, 384), ([1500], 4104, 128), ([255, 257, 0, 513, 300], 5128, 256),
                  ([128, 127, 129, 0, 1, 700], 6152, 384), ([40, 1000, 3, 64, 65, 200], 5896, 640)]
LARGER_GATE_UP = [([30] * 20, 1024, 256), (MIXED, 1280, 384), ([9] * 30, 1024, 128), ([17, 33, 0, 66, 5] * 5, 768, 640),
                  ([1500], 2048, 128), ([255, 257, 0, 513, 300], 1920, 256), ([128, 127, 129, 0, 1, 700], 2176, 384),
                  ([40, 1000, 3, 64, 65, 200], 1792, 512)]


@pytest.mark.parametrize("counts,N,K", LARGER_PRODUCT)
def test_larger_product_exact(ep, counts, N, K):
    gen = torch.Generator(device="cuda").manual_seed(21)
    off = offsets(counts, 3)
    M = off[-1] + 7
    rows, x, w, sw, w64 = exact_inputs(M, len(counts), N, K, gen)
    log(f"[product] counts={counts[:6]} N={N} K={K}")
    out, st = product(ep, rows, off, w, sw, M, N)
    assert st == 0
    want = R.grouped64(x, off, w64)
    assert torch.equal(out[3:off[-1]], want[3:off[-1]].float().bfloat16())
    assert (out[:3] == -7).all() and (out[off[-1]:] == -7).all()
    # a NaN row and a NaN weight row: nothing else moves
    bad = min(off[1] if counts[0] else off[2], off[-1] - 1)
    g = next(i for i, c in enumerate(counts) if c and off[i] <= bad < off[i + 1])
    rows2, w2 = rows.clone(), w.clone()
    rows2[bad, K - 1] = 0x7F
    w2[g, N - 1, 0] = 0xFF
    dirty, _ = product(ep, rows2, off, w2, sw, M, N)
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[bad] = False
    ok[off[g]:off[g + 1], N - 1] = False
    assert torch.equal(out[ok], dirty[ok])
    assert torch.isnan(dirty[bad]).all() and torch.isnan(dirty[off[g]:off[g + 1], N - 1]).all()


@pytest.mark.parametrize("counts,F,K", LARGER_GATE_UP)
def test_larger_gate_up_exact(ep, counts, F, K):
    gen = torch.Generator(device="cuda").manual_seed(22)
    off = offsets(counts, 3)
    M = off[-1] + 7
    rows, x, w, sw, _ = exact_inputs(M, len(counts), 2 * F, K, gen)
    sw = sw * 2.0 ** -6
    w64 = R.weights64(w.view(torch.float8_e4m3fn), sw)
    log(f"[gate_up] counts={counts[:6]} F={F} K={K}")
    out, st = gate_up(ep, rows, off, w, sw, M, F)
    assert st == 0
    y = R.grouped64(x, off, w64)[3:off[-1]]
    g, u = y[:, :F], y[:, F:]
    h = g / (1 + torch.exp(-g)) * u
    big = g.abs().view(g.shape[0], -1, 128).amax(2)
    R.assert_rows8(out[3:off[-1]], h, (big + 6) * R.U32, "out_rows")
    assert (out[:3] == 0xA5).all() and (out[off[-1]:] == 0xA5).all()
    # a NaN row, and a NaN weight row (the last up): nothing else moves
    bad = min(off[1] if counts[0] else off[2], off[-1] - 1)
    e = next(i for i, c in enumerate(counts) if c and off[i] <= bad < off[i + 1])
    rows2, w2 = rows.clone(), w.clone()
    rows2[bad, K - 1] = 0x7F
    w2[e, 2 * F - 1, 0] = 0xFF
    dirty, _ = gate_up(ep, rows2, off, w2, sw, M, F)
    ok = torch.ones_like(out, dtype=torch.bool)
    ok[bad] = False
    ok[off[e]:off[e + 1], F - 128:F] = False     # the block that shares its scale
    ok[off[e]:off[e + 1], F + F // 32 - 4:F + F // 32] = False
    assert torch.equal(out[ok], dirty[ok])
    assert ((dirty[bad, :F] & 0x7F) == 0x7F).all()
    assert ((dirty[off[e]:off[e + 1], F - 1] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("counts,N,K", [([40, 30, 25, 0, 50, 8] * 3, 2056, 1792), ([700, 600, 300], 5128, 1792)])
def test_larger_product_random(ep, counts, N, K):
    gen = torch.Generator(device="cuda").manual_seed(23)
    off = offsets(counts)
    M, G = off[-1], len(counts)
    rows, x = R.make_rows(torch.randn(M, K, device="cuda", generator=gen) * 3)
    w, sw, w64 = R.make_weights(G, N, K, gen)
    out, st = product(ep, rows, off, w, sw, M, N)
    assert st == 0
    want = R.grouped64(x, off, w64)
    R.assert_close(out, want, want.abs() * R.U_BF16 + R.mfma_bound(x, off, w64), "out")
    assert float((out.double() - want).norm() / want.norm()) <= R.U_BF16 + 2.0 ** -13


def test_larger_bad_offsets_are_reported(ep):
    """Rows beyond M are skipped by the middle and the big tiles too, and
    offsets out of order write nothing outside the outputs."""
    gen = torch.Generator(device="cuda").manual_seed(24)
    for counts, N, K in [([30] * 20, 1304, 512), ([700, 0, 800], 4104, 128)]:
        off = offsets(counts)
        M = off[-1]
        rows, x, w, sw, w64 = exact_inputs(M, len(counts), N, K, gen)
        guard = torch.full((3 * M, N), -7.0, dtype=torch.bfloat16, device="cuda")
        st = i32([0])
        ep.ep_expert_product(rows, i32(off[:-1] + [M + 1]), w, sw, guard[M:2 * M], st)
        assert int(st) == 3
        assert torch.equal(guard[M:2 * M], R.grouped64(x, off, w64).float().bfloat16())
        swapped = list(off)
        swapped[1], swapped[2] = swapped[2], swapped[1] - 20
        st = i32([0])
        ep.ep_expert_product(rows, i32(swapped), w, sw, guard[M:2 * M], st)
        assert int(st) == 1
        assert (guard[:M] == -7).all() and (guard[2 * M:] == -7).all()


def test_offsets_that_count_rows_many_times(ep):
    """Offsets that go up and down name more rows than there are: the call
    reports them, ends, and writes nothing outside its output."""
    gen = torch.Generator(device="cuda").manual_seed(25)
    M, G, N, K = 1500, 20, 4104, 128
    rows, x, w, sw, w64 = exact_inputs(M, G, N, K, gen)
    guard = torch.full((3 * M, N), -7.0, dtype=torch.bfloat16, device="cuda")
    for m in (M, 600):     # big tiles, middle tiles
        st = i32([0])
        ep.ep_expert_product(rows[:m], i32([0, m] * (G // 2) + [0]), w, sw, guard[M:M + m], st)
        assert int(st) == 1
        assert (guard[:M] == -7).all() and (guard[M + M:] == -7).all()
    guard[M:] = -7.0
    ep.ep_expert_product(rows[:m], i32([0, m] * (G // 2) + [0]), w, sw, guard[M:M + m], i32([0]))
    assert (guard[M + m:] == -7).all()


@pytest.mark.parametrize("which", ["product", "gate_up"])
def test_many_tiles_a_workgroup(ep, which):
    """More tiles than the GPU has CUs, so that workgroups go from one to the
    next: whole, ragged and short ones of several groups."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    counts, K = [1000, 0, 256, 3, 2817, 511], 256
    off = offsets(counts, 2)
    M = off[-1] + 5
    N = 5896 if which == "product" else 2 * 2944
    rows, x, w, sw, w64 = exact_inputs(M, len(counts), N, K, gen)
    inside = slice(2, off[-1])
    for _ in range(2):
        if which == "product":
            out, st = product(ep, rows, off, w, sw, M, N)
            want = R.grouped64(x, off, w64)
            assert torch.equal(out[inside], want[inside].float().bfloat16())
            assert (out[:2] == -7).all() and (out[off[-1]:] == -7).all()
        else:
            out, st = gate_up(ep, rows, off, w, sw * 2.0 ** -6, M, N // 2)
            y = R.grouped64(x, off, w64 * 2.0 ** -6)[inside]
            g, u = y[:, :N // 2], y[:, N // 2:]
            h = g / (1 + torch.exp(-g)) * u
            big = g.abs().view(g.shape[0], -1, 128).amax(2)
            R.assert_rows8(out[inside], h, (big + 6) * R.U32, "out_rows")
            assert (out[:2] == 0xA5).all() and (out[off[-1]:] == 0xA5).all()
        assert st == 0


@pytest.mark.parametrize("which", ["product", "gate_up"])
@pytest.mark.parametrize("counts,N,K", [([20, 70, 3], 256, 256), ([30] * 20, 2048, 512),
                                        ([1000, 0, 256, 3, 2817, 511], 5888, 256)])
def test_infinite_scales_stay_in_their_rows(ep, which, counts, N, K):
    """An infinite scale in the last block of K of some rows, or of one expert's
    weights, changes no other row, in small, middle and big tiles; of the last
    there are more than CUs, so that a workgroup goes from a tile with such a
    scale to one without."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    off = offsets(counts, 2)
    M, G = off[-1] + 5, len(counts)
    rows, x, w, sw, _ = exact_inputs(M, G, N, K, gen)
    f, n = (product, N) if which == "product" else (gate_up, N // 2)
    log(f"[infinite scales] {which} counts={counts[:6]} N={N} K={K}")
    clean, st = f(ep, rows, off, w, sw, M, n)
    assert st == 0
    place = torch.full((M,), -1, device="cuda")
    for g in range(G):
        place[off[g]:off[g + 1]] = torch.arange(counts[g], device="cuda")
    # of every third 256 rows of an expert, the second half of each 64
    bad = (place >= 0) & (place // 256 % 3 == 0) & (place % 64 >= 32) if max(counts) >= 64 else place == 29
    assert bad.any()
    rows2 = rows.clone()
    inf = torch.full((1,), float("inf"), device="cuda").view(torch.uint8)
    rows2[bad, K + K // 32 - 4:K + K // 32] = inf
    dirty, st = f(ep, rows2, off, w, sw, M, n)
    assert st == 0
    assert torch.equal(clean[~bad].view(torch.uint8), dirty[~bad].view(torch.uint8))
    if which == "product":
        assert not torch.isfinite(dirty[bad]).any()
    for g in range(min(G, 6)):
        sw2 = sw.clone()
        sw2[g, :, -1] = float("inf")
        dirty, st = f(ep, rows, off, w, sw2, M, n)
        assert st == 0
        other = torch.ones(M, dtype=torch.bool, device="cuda")
        other[off[g]:off[g + 1]] = False
        assert torch.equal(clean[other].view(torch.uint8), dirty[other].view(torch.uint8)), f"expert {g}"
        if which == "product":
            assert not torch.isfinite(dirty[~other]).any()


def test_weights_as_float8_and_many_groups(ep):
    """1024 experts, most without rows; codes passed as float8."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    G, N, K = 1024, 128, 128
    r = np.random.RandomState(8)
    counts = np.zeros(G, np.int64)
    for e in r.randint(0, G, 400):
        counts[e] += 1
    off = offsets(counts)
    M = off[-1] + 3
    rows, x, w, sw, w64 = exact_inputs(M, G, N, K, gen)
    out, st = product(ep, rows, off, w.view(torch.float8_e4m3fn), sw, M, N)
    assert st == 0
    assert torch.equal(out[:off[-1]], R.grouped64(x, off, w64)[:off[-1]].float().bfloat16())
    out, st = gate_up(ep, rows, off, w.view(torch.float8_e4m3fn).repeat(1, 2, 1).contiguous(),
                      sw.repeat(1, 2, 1).contiguous() * 2.0 ** -6, M, N)
    assert st == 0 and (out[off[-1]:] == 0xA5).all() and not (out[:off[-1], N + 4:] != 0).any()


@pytest.mark.parametrize("float8", [False, True])
def test_gate_up_of_many_groups(ep, float8):
    """1024 experts, most without rows, all with weights of their own: values."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    G, F, K = 1024, 128, 128
    r = np.random.RandomState(15)
    counts = np.bincount(r.randint(0, G, 400), minlength=G)
    off = offsets(counts)
    M = off[-1] + 3
    rows, x, w, sw, _ = exact_inputs(M, G, 2 * F, K, gen)
    sw = sw * 2.0 ** -6
    w64 = R.weights64(w.view(torch.float8_e4m3fn), sw)
    out, st = gate_up(ep, rows, off, w.view(torch.float8_e4m3fn) if float8 else w, sw, M, F)
    y = R.grouped64(x, off, w64)[:off[-1]]
    g, u = y[:, :F], y[:, F:]
    h = g / (1 + torch.exp(-g)) * u
    big = g.abs().view(g.shape[0], -1, 128).amax(2)
    assert st == 0
    R.assert_rows8(out[:off[-1]], h, (big + 6) * R.U32, "out_rows")
    assert (out[off[-1]:] == 0xA5).all()


@pytest.mark.parametrize("which", ["product", "gate_up"])
@pytest.mark.parametrize("each,N,K", [(12, 520, 128), (70, 1024, 256)])
def test_more_than_64_groups_of_larger_tiles(ep, which, each, N, K):
    """Middle and big tiles whose groups take a wavefront several looks: 200
    experts, every third without rows, the last with many."""
    gen = torch.Generator(device="cuda").manual_seed(16)
    counts = [0 if g % 3 == 1 else each + g % 29 for g in range(199)] + [900]
    off = offsets(counts, 1)
    M, n = off[-1] + 2, N if which == "product" else 512
    rows, x, w, sw, _ = exact_inputs(M, 200, n if which == "product" else 2 * n, K, gen)
    inside = slice(1, off[-1])
    if which == "product":
        out, st = product(ep, rows, off, w, sw, M, n)
        want = R.grouped64(x, off, R.weights64(w.view(torch.float8_e4m3fn), sw))
        assert torch.equal(out[inside], want[inside].float().bfloat16())
        assert (out[:1] == -7).all() and (out[off[-1]:] == -7).all()
    else:
        sw = sw * 2.0 ** -6
        out, st = gate_up(ep, rows, off, w, sw, M, n)
        y = R.grouped64(x, off, R.weights64(w.view(torch.float8_e4m3fn), sw))[inside]
        g, u = y[:, :n], y[:, n:]
        h = g / (1 + torch.exp(-g)) * u
        big = g.abs().view(g.shape[0], -1, 128).amax(2)
        R.assert_rows8(out[inside], h, (big + 6) * R.U32, "out_rows")
        assert (out[:1] == 0xA5).all() and (out[off[-1]:] == 0xA5).all()
    assert st == 0


def test_same_bits_each_time_and_graph(ep):
    gen = torch.Generator(device="cuda").manual_seed(9)
    counts, H, F = [0, 12, 200, 7], 512, 256
    off = offsets(counts)
    M, G = off[-1], len(counts)
    rows, _ = R.make_rows(torch.randn(M, H, device="cuda", generator=gen))
    w1, s1, _ = R.make_weights(G, 2 * F, H, gen)
    w2, s2, _ = R.make_weights(G, H, F, gen)
    d_off, st = i32(off), i32([0])
    inner = torch.zeros(M, R.row_bytes(F), dtype=torch.uint8, device="cuda")
    out = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")

    def both():
        ep.ep_expert_gate_up(rows, d_off, w1, s1, inner, st)
        ep.ep_expert_product(inner, d_off, w2, s2, out, st)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in range(3):
        gen.manual_seed(20 + seed)
        new, _ = R.make_rows(torch.randn(M, H, device="cuda", generator=gen))
        rows.copy_(new)
        d_off.copy_(i32(offsets([seed * 3, 12 - seed, 200, 2])))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        both()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and int(st) == 0


def test_other_stream(ep):
    gen = torch.Generator(device="cuda").manual_seed(10)
    off = offsets([20, 90])
    rows, x, w, sw, w64 = exact_inputs(110, 2, 136, 256, gen)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, st = product(ep, rows, off, w, sw, 110, 136)
    s.synchronize()
    assert st == 0 and torch.equal(out, R.grouped64(x, off, w64).float().bfloat16())


def test_refusals_by_the_binding(ep):
    gen = torch.Generator(device="cuda").manual_seed(11)
    rows, _, w, sw, _ = exact_inputs(8, 2, 256, 256, gen)
    out = torch.empty(8, 256, dtype=torch.bfloat16, device="cuda")
    ok = dict(rows=rows, group_offset=i32([0, 4, 8]), w=w, w_scale=sw, out=out, dev_status=i32([0]))
    ep.ep_expert_product(**ok)
    for bad in [dict(rows=rows[:, :256].contiguous()), dict(rows=rows.cpu()), dict(rows=None),
                dict(group_offset=i32([0, 8])), dict(group_offset=i32([0, 4, 8]).long()), dict(w=w.float()),
                dict(w=w[0]), dict(w_scale=sw[:, :1].contiguous()), dict(w_scale=sw.double()), dict(out=out[:4]),
                dict(out=out.float()), dict(dev_status=None)]:
        with pytest.raises(ValueError):
            ep.ep_expert_product(**{**ok, **bad})
    for n in (100, 4):
        with pytest.raises(ep.EpError):
            ep.ep_expert_product(rows, i32([0, 4, 8]), w[:, :n].contiguous(), sw[:, :1].contiguous(),
                                 out[:, :n].contiguous(), i32([0]))
    with pytest.raises(ep.EpError):      # the gate's halves are whole blocks
        ep.ep_expert_gate_up(rows, i32([0, 4, 8]), w[:, :128].contiguous(), sw[:, :1].contiguous(), rows, i32([0]))
