"""ep_route and its backward against 64 bits.

Tolerances: exp(l - top) is off by two roundings and one of l - top, which
scales with it; a lane adds up to 64 of them, then six steps: REL(span) for the
weights, lse's logarithm the same."""

import pytest
import torch

import operator_refs as R
from gpu_helpers import log

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 4, 2), (3, 5, 5), (17, 16, 2), (128, 16, 2), (65, 20, 3), (40, 33, 7), (31, 60, 6),
         (50, 97, 8), (129, 128, 8), (77, 200, 31), (128, 256, 8), (300, 256, 32), (45, 257, 8), (33, 384, 6),
         (20, 777, 9), (19, 1024, 8), (7, 1500, 4), (9, 4096, 32), (4100, 64, 4), (16384, 256, 8)]


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def rel(span):
    return (2 * span + 80) * R.U32


def forward(ep, logits, mask, k, mode, stats=True, ws=None, stream=None):
    T, E = logits.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(topk_idx=torch.full((T, k), -77, **i32), topk_w=torch.full((T, k), float("nan"), device="cuda"),
             num_tokens_per_expert=torch.full((E,), -7, **i32) if stats else None,
             num_tokens=torch.full((1,), -7, **i32) if stats else None,
             lse=torch.full((T,), float("nan"), device="cuda"),
             balance_loss=torch.full((1,), float("nan"), device="cuda") if stats else None)
    if stats and ws is None:
        ws = torch.zeros(ep.ep_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    ep.ep_route(logits, mask, mode, **o, workspace=ws, stream=stream)
    return o


def keep_of(logits, mask):
    return torch.ones(logits.shape[0], dtype=torch.bool, device="cuda") if mask is None else mask != 0


def check(o, logits, mask, k, mode):
    keep = keep_of(logits, mask)
    idx, w, counts, n, lse, loss, _ = R.route64(logits, keep, k, mode)
    assert torch.equal(o["topk_idx"], idx)
    l = logits.double()[keep]
    l = l[torch.isfinite(l)]
    span = float((l.max() - l.min())) if l.numel() else 0.0
    R.assert_close(o["topk_w"], w, w * rel(span) + 2.0 ** -126, "topk_w")
    R.assert_close(o["lse"], lse, torch.nan_to_num(lse.abs(), posinf=0.0) * 2 * R.U32 + rel(span), "lse")
    if o["balance_loss"] is not None:
        assert torch.equal(o["num_tokens_per_expert"], counts)
        assert int(o["num_tokens"]) == n
        # the sums over tokens: a group's, then its workgroup's, in float
        T = logits.shape[0]
        R.assert_close(o["balance_loss"][0], loss, loss * (rel(span) + (T / 1024 + 16) * R.U32), "balance_loss")


def make(T, E, half, seed=0, masked=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = 2 * torch.randn(T, E, device="cuda", generator=g)
    mask = None
    if masked:
        mask = (torch.rand(T, device="cuda", generator=g) < 0.7).to(torch.uint8) * 3
        logits[mask == 0] = float("nan")
        logits[(mask == 0).nonzero()[::2, 0]] = float("inf")
    return logits.bfloat16() if half else logits, mask


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("half,mode,masked", [(False, 1, False), (True, 0, True)])
def test_forward(ep, T, E, k, half, mode, masked):
    logits, mask = make(T, E, half, masked=masked)
    log(f"[route] T={T} E={E} k={k} half={half} mode={mode}")
    check(forward(ep, logits, mask, k, mode), logits, mask, k, mode)
    check(forward(ep, logits, mask, k, mode, stats=False), logits, mask, k, mode)


@pytest.mark.parametrize("E", [16, 200, 600])
def test_ties_go_to_the_lowest_expert(ep, E):
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randint(-1, 2, (64, E), device="cuda", generator=g).float()
    logits[0] = 0.5
    logits[1] = -0.0
    logits[1, ::2] = 0.0
    o = forward(ep, logits, None, 8, 1)
    check(o, logits, None, 8, 1)
    assert o["topk_idx"][0].tolist() == list(range(8))
    assert o["topk_idx"][1].tolist() == list(range(8))


@pytest.mark.parametrize("E", [12, 300])
@pytest.mark.parametrize("mode", [0, 1])
def test_masked_experts(ep, E, mode):
    """-inf logits are no choice; a row of them alone has none, weights and
    probabilities zero, and still counts as a token."""
    k = 6
    logits, _ = make(9, E, False, 4)
    logits[0] = float("-inf")
    logits[1, 3:] = float("-inf")
    logits[2, 5:] = float("-inf")
    logits[3, 1:] = float("-inf")
    logits[4] = torch.finfo(torch.float32).min      # the type's lowest value is a number
    logits[4, 2] = 0.0
    logits[5, :5] = float("-inf")
    o = forward(ep, logits, None, k, mode)
    check(o, logits, None, k, mode)
    assert (o["topk_idx"][0] == -1).all() and (o["topk_w"][0] == 0).all()
    assert o["lse"][0] == float("-inf")
    assert (o["topk_idx"][1] >= 0).sum() == 3
    assert int(o["num_tokens"]) == 9
    gl = torch.ones(1, device="cuda")
    gw = torch.ones(9, k, device="cuda")
    dl = torch.full_like(logits, float("nan"))
    ep.ep_route_backward(logits, None, mode, o["topk_idx"], o["topk_w"], o["num_tokens_per_expert"],
                         o["num_tokens"], o["lse"], gw, gl, dl)
    assert torch.isfinite(dl).all() and (dl[0] == 0).all() and (dl[1, 3:] == 0).all()


@pytest.mark.parametrize("E", [12, 300])
def test_nan_and_inf_logits_show(ep, E):
    logits, _ = make(6, E, False, 5)
    logits[1, 4] = float("nan")
    logits[3, 7] = float("inf")
    o = forward(ep, logits, None, 4, 1)
    for t in (1, 3):
        assert torch.isnan(o["topk_w"][t]).all() and torch.isnan(o["lse"][t])
    assert 4 not in o["topk_idx"][1].tolist()
    assert torch.isnan(o["balance_loss"]).all()
    good = [0, 2, 4, 5]
    assert torch.isfinite(o["topk_w"][good]).all()


def test_all_padded_and_empty(ep):
    logits = torch.full((5, 24), float("nan"), device="cuda")
    o = forward(ep, logits, torch.zeros(5, dtype=torch.uint8, device="cuda"), 3, 1)
    assert (o["topk_idx"] == -1).all() and (o["topk_w"] == 0).all() and (o["num_tokens_per_expert"] == 0).all()
    assert int(o["num_tokens"]) == 0 and float(o["balance_loss"]) == 0
    o = forward(ep, torch.empty(0, 24, device="cuda"), None, 3, 1)
    assert (o["num_tokens_per_expert"] == 0).all() and float(o["balance_loss"]) == 0


def backward(ep, logits, mask, mode, o, gw, gl, out=None):
    dl = torch.full_like(logits, float("nan")) if out is None else out
    ep.ep_route_backward(logits, mask, mode, o["topk_idx"], o["topk_w"], o["num_tokens_per_expert"],
                         o["num_tokens"], o["lse"], gw, gl, dl)
    return dl


def check_back(dl, logits, mask, k, mode, gw, gl):
    """Every part of a logit's gradient in magnitude, times the roundings of
    p = exp(l - lse) and of sums over up to 64 + 6 terms, and the type's own."""
    keep = keep_of(logits, mask)
    idx, w, counts, n, lse, _, p = R.route64(logits, keep, k, mode)
    want = torch.where(keep[:, None], R.route_back64(p, idx, w, counts, n, mode, gw, gl), 0.0)
    parts = R.route_back64(-p.abs(), idx, w, -counts, n, mode, None, gl).abs()
    m = max(n, 1)
    d = torch.zeros(logits.shape[1], dtype=torch.float64, device="cuda")
    if gl is not None:
        d = (gl.double() * logits.shape[1] * counts / (m * m * k)).abs()
    parts = p * (d + (p * d).sum(1, keepdim=True))
    if gw is not None:
        z = (gw.double() * w).abs()
        S = z.sum(1, keepdim=True)
        parts = parts + p * S
        parts = parts.scatter_add(1, idx.clamp_min(0).long(), z + w * S)
    l = torch.where(keep[:, None], logits.double(), 0.0)
    span = float((lse.abs().max() + l.abs().max())) if l.numel() else 0.0
    tol = parts * (rel(span) + 90 * R.U32) + 2.0 ** -126
    if logits.dtype == torch.bfloat16:
        tol = tol + want.abs() * R.U_BF16
    R.assert_close(dl, want, tol, "grad_logits")


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("half,mode,masked,parts", [(False, 1, True, "both"), (True, 0, False, "both"),
                                                    (False, 0, True, "gates"), (False, 1, False, "loss")])
def test_backward(ep, T, E, k, half, mode, masked, parts):
    logits, mask = make(T, E, half, 6, masked)
    o = forward(ep, logits, mask, k, mode)
    g = torch.Generator(device="cuda").manual_seed(7)
    gw = torch.randn(T, k, device="cuda", generator=g) if parts != "loss" else None
    gl = torch.full((1,), 0.3, device="cuda") if parts != "gates" else None
    log(f"[route backward] T={T} E={E} k={k} {parts}")
    check_back(backward(ep, logits, mask, mode, o, gw, gl), logits, mask, k, mode, gw, gl)


@pytest.mark.parametrize("T,E,k", [(40, 20, 3), (33, 256, 8), (9, 777, 9)])
@pytest.mark.parametrize("mode", [0, 1])
def test_backward_far_from_zero(ep, T, E, k, mode):
    """Softmax does not change when a token's logits move together: logits of
    whole 256ths around 8192, held exactly, have the gradients of those around
    0, within the tolerance of those (lse, held in float, is itself off by up to
    2^-11 there)."""
    logits, _ = make(T, E, False, 19)
    logits = (logits * 256).round() / 256
    far = logits + 8192.0
    assert torch.equal(far - 8192.0, logits)
    o = forward(ep, far, None, k, mode)
    g = torch.Generator(device="cuda").manual_seed(20)
    gw, gl = torch.randn(T, k, device="cuda", generator=g), torch.full((1,), 0.3, device="cuda")
    assert torch.equal(o["topk_idx"], R.route64(logits, keep_of(logits, None), k, mode)[0])
    check_back(backward(ep, far, None, mode, o, gw, gl), logits, None, k, mode, gw, gl)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("E,k", [(12, 3), (256, 8), (300, 5)])
def test_rows_of_the_lowest_value(ep, E, k, half, mode):
    """A token whose logits are all the type's lowest value, or all but some
    that are -inf, has equal probabilities, as with logits of zero."""
    kind = torch.bfloat16 if half else torch.float32
    T = 5
    logits, _ = make(T, E, half, 21)
    logits[1:4] = torch.finfo(kind).min
    logits[2, 1::2] = float("-inf")
    zero = logits.clone()
    zero[1:4] = 0.0
    zero[2, 1::2] = float("-inf")
    o = forward(ep, logits, None, k, mode)
    same = forward(ep, zero, None, k, mode)
    for n in ("topk_idx", "topk_w", "num_tokens_per_expert", "balance_loss"):
        assert torch.equal(o[n], same[n]), n
    gw, gl = torch.ones(T, k, device="cuda"), torch.full((1,), 0.3, device="cuda")
    gw[:, 0] = -2.0
    near = zero.clamp_min(-200.0)     # exp(-200) is no more than -inf's in float, and a finite span
    check_back(backward(ep, logits, None, mode, o, gw, gl), near, None, k, mode, gw, gl)


def test_backward_in_place(ep):
    logits, mask = make(200, 48, False, 8, True)
    keep = logits.clone()
    o = forward(ep, logits, mask, 5, 1)
    gw, gl = torch.ones(200, 5, device="cuda"), torch.ones(1, device="cuda")
    backward(ep, logits, mask, 1, o, gw, gl, out=logits)
    check_back(logits, keep, mask, 5, 1, gw, gl)


@pytest.mark.parametrize("mode", [0, 1])
def test_backward_against_differences(ep, mode):
    """sum(c * topk_w) + balance_loss in 64 bits, with the choices held, along
    random directions: the central difference of step 1e-4 is off by about
    1e-8, the gradients by float's roundings."""
    T, E, k, e = 7, 20, 3, 1e-4
    logits, _ = make(T, E, False, 9)
    o = forward(ep, logits, None, k, mode)
    g = torch.Generator(device="cuda").manual_seed(10)
    c = torch.randn(T, k, device="cuda", generator=g)
    dl = backward(ep, logits, None, mode, o, c, torch.ones(1, device="cuda")).double()
    idx, f = o["topk_idx"].long(), o["num_tokens_per_expert"].double() / (T * k)

    def loss(l):
        p = torch.softmax(l, 1)
        w = p.gather(1, idx)
        if mode:
            w = w / w.sum(1, keepdim=True)
        return (c.double() * w).sum() + E * (f * p.mean(0)).sum()

    for _ in range(4):
        u = torch.randn(T, E, device="cuda", generator=g).double()
        num = (loss(logits.double() + e * u) - loss(logits.double() - e * u)) / (2 * e)
        assert abs(float(num - (dl * u).sum())) <= float((dl * u).abs().sum()) * 1e-5 + 1e-6


def test_one_workspace_many_calls_and_a_graph(ep):
    """One workspace serves calls of several sizes in turn; the results are the
    same bits each time; captured and replayed with eager calls between."""
    T, E, k = 500, 256, 8
    ws = torch.zeros(ep.ep_route_workspace_bytes(4000, 1024), dtype=torch.uint8, device="cuda")
    first = None
    for T_, E_ in [(T, E), (4000, 1024), (3, 16), (T, E)]:
        logits, mask = make(T_, E_, False, 11, True)
        o = forward(ep, logits, mask, k, 1, ws=ws)
        check(o, logits, mask, k, 1)
        if (T_, E_) == (T, E):
            if first is not None:
                assert all(torch.equal(first[n], o[n]) for n in o)
            first = o
    logits, mask = make(T, E, False, 12, True)
    ws2 = torch.zeros(ep.ep_route_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    gw, gl, dl = torch.ones(T, k, device="cuda"), torch.ones(1, device="cuda"), torch.empty_like(logits)
    o = forward(ep, logits, mask, k, 1, ws=ws2)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ep.ep_route(logits, mask, 1, **o, workspace=ws2)
        ep.ep_route_backward(logits, mask, 1, o["topk_idx"], o["topk_w"], o["num_tokens_per_expert"],
                             o["num_tokens"], o["lse"], gw, gl, dl)
    for seed in (13, 14, 15):
        l2, m2 = make(T, E, False, seed, True)
        logits.copy_(l2)
        mask.copy_(m2)
        g.replay()
        torch.cuda.synchronize()
        check(o, logits, mask, k, 1)
        check_back(dl, logits, mask, k, 1, gw, gl)
        check(forward(ep, l2, m2, k, 0, ws=ws), l2, m2, k, 0)


@pytest.mark.parametrize("half", [False, True])
def test_logits_that_lie_between_words(ep, half):
    """Logits behind an odd offset: aligned to their type alone."""
    T, E, k = 65, 64, 4
    base, _ = make(1, T * E + 1, half, 18)
    logits = base[0, 1:].view(T, E)
    o = forward(ep, logits, None, k, 1)
    check(o, logits, None, k, 1)
    gw = torch.ones(T, k, device="cuda")
    check_back(backward(ep, logits, None, 1, o, gw, None), logits, None, k, 1, gw, None)


def test_other_stream(ep):
    logits, mask = make(1000, 256, True, 16, True)
    s = torch.cuda.Stream()
    ws = torch.zeros(ep.ep_route_workspace_bytes(1000, 256), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        o = forward(ep, logits, mask, 8, 1, ws=ws)
    s.synchronize()
    check(o, logits, mask, 8, 1)


def test_refusals_by_the_binding(ep):
    logits, mask = make(6, 16, False, 17, True)
    o = forward(ep, logits, mask, 2, 1)
    ws = torch.zeros(ep.ep_route_workspace_bytes(6, 16), dtype=torch.uint8, device="cuda")
    for bad in [dict(logits=logits.double()), dict(logits=logits.cpu()), dict(logits=logits.t()),
                dict(token_mask=mask.bool()), dict(token_mask=mask[:3]), dict(topk_idx=o["topk_idx"].long()),
                dict(topk_w=o["topk_w"][:3]), dict(topk_w=None), dict(lse=o["lse"].double()),
                dict(num_tokens_per_expert=o["num_tokens_per_expert"][:4]), dict(workspace=None)]:
        with pytest.raises(ValueError):
            ep.ep_route(**{**dict(logits=logits, token_mask=mask, mode=1, workspace=ws, **o), **bad})
    for bad in [dict(mode=2), dict(balance_loss=None), dict(workspace=ws[:64])]:
        with pytest.raises(ep.EpError):
            ep.ep_route(**{**dict(logits=logits, token_mask=mask, mode=1, workspace=ws, **o), **bad})
    with pytest.raises(ValueError):
        backward(ep, logits, mask, 1, o, torch.ones(6, 3, device="cuda"), None)
    with pytest.raises(ValueError):
        backward(ep, logits, mask, 1, {**o, "lse": None}, None, None)
