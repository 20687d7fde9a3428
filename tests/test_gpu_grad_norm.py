"""The gradients' norm and clipping against 64 bits.

Tolerances: squares and sums are double, n of them (n roundings at most); the
norm is rounded to float once.  A clipped element is off by the ratio's and the
product's rounding and by the output's own."""

import math

import pytest
import torch

from gpu_helpers import log
from operator_refs import U32, U_BF16, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def workspace(ep, n):
    return torch.zeros(ep.ep_grad_norm_workspace_bytes(n), dtype=torch.uint8, device="cuda")


def make(sizes, half, seed=0, shift=0):
    """Tensors of these sizes at odd places of one buffer a type."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + 16, device="cuda", generator=gen) * 10.0 ** (i % 5 - 3)
        t = t.bfloat16() if half(i) else t
        off = (i * 3 + shift) % 9
        out.append(t[off:off + n])
    return out


def norm64(tensors):
    return sum((t.double() ** 2).sum() for t in tensors) if tensors else torch.zeros((), dtype=torch.float64)


def run(ep, tensors, ws=None, stream=None):
    s, n = torch.full((1,), -1.0, dtype=torch.float64, device="cuda"), torch.full((1,), -1.0, device="cuda")
    ep.ep_grad_norm(tensors, s, n, workspace(ep, len(tensors)) if ws is None else ws, stream)
    return s, n


def check_norm(s, n, tensors):
    want = float(norm64(tensors))
    count = sum(t.numel() for t in tensors)
    assert abs(float(s) - want) <= want * (count + 4) * 2.0 ** -52      # ours and that of `want`
    root = math.sqrt(want)
    assert abs(float(n) - root) <= root * (U32 + (count + 4) * 2.0 ** -52) + 2.0 ** -149


def check_clip(got, t, want_ratio):
    want = t.double() * want_ratio
    step = U_BF16 if got.dtype == torch.bfloat16 else U32
    # a result below float's normal range is rounded to its own grid twice
    tol = want.abs() * (step * (1 + 4 * U32) + 3 * U32) + (2.0 ** -133 if got.dtype == torch.bfloat16 else 2.0 ** -148)
    assert_close(got, want, tol, "clipped")


SIZES = {
    "one": [1], "seven": [7], "few": [5, 1, 0, 8, 9, 16385, 3], "unit": [16384, 16383, 16385, 32768],
    "edge": [8191, 8192, 8193, 16400], "many": [(i * 37) % 301 for i in range(1000)], "tables": [3] * 128 + [40000] + [5] * 200,
    "large": [30_000_000, 11, 5_000_001], "empty": [0, 0, 0],
    "thousands": [(i * 61) % 977 for i in range(3000)], "among empty": [0] * 70 + [40000] + [0] * 200 + [7, 16384 * 3] + [0] * 64 + [5]}


@pytest.mark.parametrize("half", ["bf16", "float", "mixed"])
@pytest.mark.parametrize("name", list(SIZES))
def test_norm_and_clip(ep, name, half):
    log(f"[grad norm] {name} {half}")
    kind = {"bf16": lambda i: True, "float": lambda i: False, "mixed": lambda i: i % 3 != 1}[half]
    tensors = make(SIZES[name], kind)
    tl = ep.TensorList(tensors)
    s, n = run(ep, tensors)
    check_norm(s, n, tensors)
    norm = math.sqrt(float(s))
    before = [t.clone() for t in tensors]
    # a bound that clips, into tensors of the other type and of other alignment
    into = make(SIZES[name], lambda i: not kind(i) if i % 2 else kind(i), seed=9, shift=1)
    into_list = ep.TensorList(into)
    bound = 0.37 * norm
    ep.ep_grad_clip(tl, s, bound, into_list)
    for got, t in zip(into, before):
        check_clip(got, t, bound / norm if norm else 1.0)
    assert all(torch.equal(t, b) for t, b in zip(tensors, before))
    # a bound that does not: copied, rounded where the type is narrower
    ep.ep_grad_clip(tl, s, 2.0 * norm + 1.0, into_list)
    for got, t in zip(into, before):
        assert torch.equal(got, t.to(got.dtype))
    # in place: left as they are, then clipped
    ep.ep_grad_clip(tl, s, norm * (1 + 2.0 ** -20) + 1e-30)
    assert all(torch.equal(t, b) for t, b in zip(tensors, before))
    ep.ep_grad_clip(tl, s, bound)
    for got, t in zip(tensors, before):
        check_clip(got, t, bound / norm if norm else 1.0)


def test_outside_of_the_tensors_nothing_changes(ep):
    gen = torch.Generator(device="cuda").manual_seed(1)
    for kind in (torch.bfloat16, torch.float32):
        flat = torch.randn(100_000, device="cuda", generator=gen).to(kind)
        before = flat.clone()
        spans = [(3, 4), (7, 20), (33, 33), (50, 16450), (20_001, 60_000), (60_000, 60_009), (99_999, 100_000)]
        s, _ = run(ep, [flat[a:b] for a, b in spans])
        ep.ep_grad_clip([flat[a:b] for a, b in spans], s, 0.5 * math.sqrt(float(s)))
        inside = torch.zeros(100_000, dtype=torch.bool, device="cuda")
        for a, b in spans:
            inside[a:b] = True
        assert torch.equal(flat[~inside], before[~inside])
        assert torch.equal(flat[inside], (before[inside].float() * 0.5).to(kind))


def test_range(ep):
    """Elements whose squares leave float's range; a bound that takes all of them to
    the ends of it."""
    big = torch.full((1000,), 3e38, device="cuda")
    s, n = run(ep, [big])
    assert float(s) == pytest.approx(1000 * float(big[0]) ** 2, rel=1e-12) and math.isinf(float(n))
    ep.ep_grad_clip([big], s, 1e-3)
    assert_close(big, torch.full((1000,), 1e-3 / math.sqrt(1000), dtype=torch.float64, device="cuda"), 1e-3 / math.sqrt(1000) * 4 * U32, "big")
    small = torch.full((4096,), 1e-38, device="cuda")
    s, n = run(ep, [small])
    want = float(small[0]) * 64
    assert abs(float(n) - want) <= want * 2 * U32
    tiny = small.clone()
    ep.ep_grad_clip([tiny], s, want * 0.25)
    assert_close(tiny, small.double() * 0.25, 2.0 ** -148, "tiny")
    ep.ep_grad_clip([small], s, 0.0)
    assert (small == 0).all()
    half = torch.full((4096,), 1e30, device="cuda").bfloat16()
    s, n = run(ep, [half])
    value = float(half[0])
    ep.ep_grad_clip([half], s, 1e-30)        # a ratio of 1e-62, far below float's range
    assert_close(half, torch.full((4096,), 1e-30 / 64, dtype=torch.float64, device="cuda"), 1e-30 / 64 * (U_BF16 + 4 * U32), "half")
    assert value > 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_infinite_and_nan(ep, bad):
    tensors = make([1000, 30000, 17], lambda i: i == 1)
    tensors[1][12345] = bad
    before = [t.clone() for t in tensors]
    s, n = run(ep, tensors)
    assert math.isnan(float(n)) if math.isnan(bad) else math.isinf(float(n))
    into = [torch.zeros_like(t) for t in tensors]
    ep.ep_grad_clip(tensors, s, 1.0)
    ep.ep_grad_clip(tensors, s, 1.0, into)
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), 7.0), torch.nan_to_num(b.float(), 7.0))  # noqa: E731
    assert all(same(t, b) for t, b in zip(tensors, before))
    assert all(same(t, b) for t, b in zip(into, before))


def test_same_bits_every_time_and_from_any_workspace(ep):
    tensors = make([3_000_000, 5, 700_000, 12345], lambda i: i % 2 == 0)
    ws = workspace(ep, 4)
    first, _ = run(ep, tensors, ws)
    for _ in range(20):
        assert torch.equal(run(ep, tensors, ws)[0], first)
    assert torch.equal(run(ep, tensors, workspace(ep, 500))[0], first)
    assert int(ws[:256].sum()) == 0


def test_captured(ep):
    """Both calls in a graph, replayed with the program's own work between; 300
    tensors, so three launches each."""
    tensors = make([1000 + 7 * i for i in range(300)], lambda i: i % 2 == 0)
    tl = ep.TensorList(tensors)
    ws = workspace(ep, 300)
    s, n = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    fresh = [t.clone() for t in tensors]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ep.ep_grad_norm(tl, s, n, ws)
        ep.ep_grad_clip(tl, s, 1.0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.ep_grad_norm(tl, s, n, ws)
        ep.ep_grad_clip(tl, s, 1.0)
    for i in range(4):
        for t, f in zip(tensors, fresh):
            t.copy_(f * (i + 1))
        want_s, want_n = run(ep, tensors)
        want = [t.clone() for t in tensors]
        ep.ep_grad_clip(want, want_s, 1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, want_s) and torch.equal(n, want_n)
        assert all(torch.equal(t, w) for t, w in zip(tensors, want))


def test_two_streams(ep):
    a, b = make([4_000_000], lambda i: True, seed=1), make([4_000_000], lambda i: False, seed=2)
    want = [float(norm64(a)), float(norm64(b))]
    side = torch.cuda.Stream()
    ws, sb = workspace(ep, 1), torch.zeros(1, dtype=torch.float64, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ep.ep_grad_norm(b, sb, None, ws, side)
    sa, _ = run(ep, a)
    torch.cuda.synchronize()
    assert float(sa) == pytest.approx(want[0], rel=1e-9) and float(sb) == pytest.approx(want[1], rel=1e-9)


def test_a_list_holds_its_memory(ep):
    t = torch.ones(1000, device="cuda")
    tl = ep.TensorList([t])
    t.data = torch.zeros(1000, device="cuda")       # the list keeps what it was made for
    s, n = run(ep, tl.tensors)
    s2, _ = torch.zeros(1, dtype=torch.float64, device="cuda"), None
    ep.ep_grad_norm(tl, s2, None, workspace(ep, 1))
    assert float(s) == 1000.0 and float(s2) == 1000.0


def test_lists_without_elements(ep):
    """No table is followed where there is nothing: the C call takes NULL then."""
    import ctypes
    s, ws = torch.full((1,), -1.0, dtype=torch.float64, device="cuda"), workspace(ep, 0)
    for tensors in ([], [torch.empty(0, device="cuda")] * 3):
        tl = ep.TensorList(tensors)
        tl.c.table = None
        assert ep.lib.ep_grad_norm(ctypes.byref(tl.c), s.data_ptr(), None, ws.data_ptr(), ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert float(s) == 0.0
        s.fill_(-1.0)


def test_refusals(ep):
    t = torch.ones(64, device="cuda")
    s, n, ws = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda"), workspace(ep, 4)
    assert len(ep.TensorList([t, t.clone()])) == 2
    for bad in ([t.half()], [t.double()], [t.cpu()], [t[::2]], [t, t], [t[:10], t[9:]], [t, t.cpu()], [t.view(8, 8).t()]):
        with pytest.raises(ValueError):
            ep.ep_grad_norm(bad, s, n, ws)
    for bad in (dict(sum_squares=s.float()), dict(sum_squares=None), dict(norm=s), dict(workspace=None), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            ep.ep_grad_norm([t], **{**dict(sum_squares=s, norm=n, workspace=ws), **bad})
    with pytest.raises(ep.EpError):
        ep.ep_grad_norm([t], s, n, ws[:64])
    with pytest.raises(ValueError):
        ep.ep_grad_clip([t], s, 1.0, [t, t.clone()])
    for bad in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(into=[torch.ones(63, device="cuda")])):
        with pytest.raises(ep.EpError):
            ep.ep_grad_clip(**{**dict(tensors=[t], sum_squares=s, max_norm=1.0), **bad})
    ep.ep_grad_norm([], s, n, ws)
    assert float(s) == 0.0 and float(n) == 0.0
    ep.ep_grad_clip([], s, 1.0)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_a_tensor_of_more_than_2_to_the_31_elements(ep, kind):
    n = 2 ** 31 + 20_011
    at = [0, 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31, n - 16385, n - 1]
    flat = torch.zeros(n + 5, dtype=kind, device="cuda")
    flat[n:] = 7.0                      # behind it
    t = flat[:n]
    for i, j in enumerate(at):
        t[j] = float(i + 1)
    s, norm = run(ep, [t, torch.full((3,), 2.0, device="cuda")])
    assert float(s) == sum((i + 1) ** 2 for i in range(len(at))) + 12
    root = math.sqrt(float(s))
    ep.ep_grad_clip([t], s, root / 2)
    assert [float(t[j]) for j in at] == [(i + 1) / 2 for i in range(len(at))]
    assert (flat[n:] == 7.0).all() and int((t != 0).sum()) == len(at)
