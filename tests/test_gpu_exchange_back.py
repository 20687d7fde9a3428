"""The gradients of combine and dispatch, in both layouts, against their
definition in 64 bits.

Tolerances: a row's weight is a float sum of its choices' gates (k roundings),
its product one more and the output's rounding.  A dot product is summed over
ceil(H/512) steps of each of eight sums a lane, then three and six joins."""

import pytest
import torch

import training_refs as X
from gpu_helpers import log
from operator_refs import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def make(T, H, E, R, k, ll, seed=0, dropped=0.1, repeats=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if repeats:
        idx = torch.randint(0, E, (T, k), device="cuda", generator=g)
    else:
        idx = torch.rand(T, E, device="cuda", generator=g).argsort(1)[:, :k]
    idx = torch.where(torch.rand(T, k, device="cuda", generator=g) < dropped, -1, idx).int().contiguous()
    if T > 2:
        idx[T // 2] = -1          # a padded token
    slot, n = X.rows_of(T, E, R, k, idx, ll)
    return dict(f=f, idx=idx, w=torch.rand(T, k, device="cuda", generator=g) + 0.1, slot=slot.cuda(), n=n, gen=g)


def combine64(T, H, E, R, k, ll, d, y, grad_out, cap):
    grad_y = torch.full((cap, H), float("nan"), dtype=torch.float64)
    grad_w = torch.zeros(T, k, dtype=torch.float64)
    mag = torch.zeros(T, k, dtype=torch.float64)
    y, grad_out, w = y.double().cpu(), grad_out.double().cpu(), d["w"].double().cpu()
    for t, s, js in X.served(T, E, R, k, d["idx"], d["slot"], ll):
        grad_y[s] = sum(w[t, j] for j in js) * grad_out[t]
        grad_w[t, js] = (grad_out[t] * y[s]).sum()
        mag[t, js] = (grad_out[t] * y[s]).abs().sum()
    return grad_y.cuda(), grad_w.cuda(), mag.cuda()


SHAPES = [(1, 8, 1, 1, 1), (1, 8, 8, 4, 8), (3, 72, 16, 4, 3), (5, 512, 16, 16, 4), (37, 520, 64, 8, 8), (9, 1024, 12, 3, 5),
          (4, 1032, 64, 64, 8), (130, 256, 32, 32, 2), (2, 7168, 256, 32, 8), (6, 8200, 64, 2, 32), (3, 20000, 8, 4, 2)]


@pytest.mark.parametrize("ll", [False, True])
@pytest.mark.parametrize("T,H,E,R,k", SHAPES)
def test_combine(ep, T, H, E, R, k, ll):
    log(f"[combine back] T={T} H={H} E={E} R={R} k={k} ll={ll}")
    d = make(T, H, E, R, k, ll)
    cap = d["n"] + 3
    y, grad_out = d["f"](cap, H).bfloat16(), d["f"](T, H).bfloat16()
    grad_y = torch.full((cap, H), 77.0, dtype=torch.bfloat16, device="cuda")
    grad_w = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
    s = ep.shape(T, H, E, R, k)
    call(s, y, d["idx"], d["w"], d["slot"], grad_out, grad_y, grad_w, st)
    assert int(st) == 0
    want_y, want_w, mag = combine64(T, H, E, R, k, ll, d, y, grad_out, cap)
    none = torch.isnan(want_y[:, 0])
    assert (grad_y[none] == 77.0).all() and int(none.sum()) == 3
    assert_close(grad_y[~none], want_y[~none], X.bf16_tol(want_y[~none], want_y[~none].abs() * (k + 1) * X.U32), "grad_y")
    assert_close(grad_w, want_w, mag * (-(-H // 512) + 12) * X.U32, "grad_w")
    # each alone, and in the place of y
    only_y, only_w = torch.full_like(grad_y, 77.0), torch.full_like(grad_w, float("nan"))
    call(s, None, d["idx"], d["w"], d["slot"], grad_out, only_y, None, st)
    call(s, y, d["idx"], d["w"], d["slot"], grad_out, None, only_w, st)
    assert torch.equal(only_y, grad_y) and torch.equal(only_w, grad_w)
    inside = y.clone()
    only_w.fill_(float("nan"))
    call(s, inside, d["idx"], d["w"], d["slot"], grad_out, inside, only_w, st)
    assert torch.equal(inside[~none], grad_y[~none]) and torch.equal(inside[none], y[none])
    assert torch.equal(only_w, grad_w) and int(st) == 0


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("ll", [False, True])
@pytest.mark.parametrize("T,H,E,R,k", SHAPES)
def test_dispatch(ep, T, H, E, R, k, ll, other):
    log(f"[dispatch back] T={T} H={H} E={E} R={R} k={k} ll={ll} other={other}")
    d = make(T, H, E, R, k, ll, seed=1)
    cap = d["n"] + 3
    rows = d["f"](cap, H).bfloat16()
    rows[d["n"]:] = float("nan")
    gates = d["f"](cap) if ll else d["f"](cap, k)
    add = d["f"](T, H).bfloat16() if other else None
    grad_x = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    grad_w = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = ep.ep_dispatch_ll_backward if ll else ep.ep_dispatch_backward
    s = ep.shape(T, H, E, R, k)
    call(s, d["idx"], d["slot"], rows, gates, add, grad_x, grad_w, st)
    assert int(st) == 0
    want = torch.zeros(T, H, dtype=torch.float64) if add is None else add.double().cpu()
    mag = want.abs()
    want_w = torch.zeros(T, k)
    r64, g = rows.double().cpu(), gates.cpu()
    for t, s_, js in X.served(T, E, R, k, d["idx"], d["slot"], ll):
        want[t] += r64[s_]
        mag[t] += r64[s_].abs()
        for j in js:
            want_w[t, j] = g[s_] if ll else g[s_, j]
    assert_close(grad_x, want.cuda(), X.bf16_tol(want, mag * (k + 1) * X.U32).cuda(), "grad_x")
    assert torch.equal(grad_w.cpu(), want_w)
    # without gates; in the place of the other gradient
    again = torch.full_like(grad_x, float("nan")) if add is None else add.clone()
    call(s, d["idx"], d["slot"], rows, None, None if add is None else again, again, None, st)
    assert torch.equal(again, grad_x) and int(st) == 0


@pytest.mark.parametrize("ll", [False, True])
def test_an_expert_named_twice(ep, ll):
    T, H, E, R, k = 40, 264, 6, 2, 6
    d = make(T, H, E, R, k, ll, seed=3, repeats=True)
    y, grad_out = d["f"](d["n"], H).bfloat16(), d["f"](T, H).bfloat16()
    grad_y, grad_w = torch.empty_like(y), torch.empty(T, k, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
    call(ep.shape(T, H, E, R, k), y, d["idx"], d["w"], d["slot"], grad_out, grad_y, grad_w, st)
    want_y, want_w, mag = combine64(T, H, E, R, k, ll, d, y, grad_out, d["n"])
    assert int(st) == 0
    assert_close(grad_y, want_y, X.bf16_tol(want_y, want_y.abs() * (k + 1) * X.U32), "grad_y")
    assert_close(grad_w, want_w, mag * (-(-H // 512) + 12) * X.U32, "grad_w")


@pytest.mark.parametrize("ll", [False, True])
def test_gradients_of_the_calls_themselves(ep, ll):
    """Against the forward calls: the library's dispatch and combine are linear in
    their rows and (combine) in the gates, so <grad, step> is the step's effect."""
    T, H, E, R, k = 200, 512, 32, 8, 4
    d = make(T, H, E, R, k, ll, seed=4)
    s = ep.shape(T, H, E, R, k)
    buf = ep.BuffersLL(s) if ll else ep.Buffers(s)
    buf.layout(d["idx"])
    slot = buf.expert_slot if ll else buf.send_slot
    assert torch.equal(slot, d["slot"])
    n, cap = d["n"], buf.capacity_rows
    # small whole numbers and powers of two: nothing is rounded
    whole = lambda *sh: torch.randint(-4, 5, sh, device="cuda", generator=d["gen"])  # noqa: E731
    y, grad_out = whole(cap, H).bfloat16(), whole(T, H).bfloat16()
    w = 2.0 ** torch.randint(-2, 1, (T, k), device="cuda", generator=d["gen"]).float()
    grad_y, grad_w = torch.zeros_like(y), torch.empty_like(w)
    call = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
    call(s, y, d["idx"], w, slot, grad_out, grad_y, grad_w, buf.dev_status)
    step = whole(cap, H).bfloat16()
    buf.combine(step, d["idx"], w)
    assert (grad_y[:n].double() * step[:n].double()).sum() == (grad_out.double() * buf.out.double()).sum()
    buf.combine(y, d["idx"], w)
    assert (grad_w.double() * w.double()).sum() == (grad_out.double() * buf.out.double()).sum()
    x = whole(T, H).bfloat16()
    buf.dispatch(x, d["idx"], w)
    rows = whole(cap, H).bfloat16()
    gates = whole(cap).float() if ll else whole(cap, k).float()
    grad_x, grad_g = torch.empty_like(x), torch.empty_like(w)
    call = ep.ep_dispatch_ll_backward if ll else ep.ep_dispatch_backward
    call(s, d["idx"], slot, rows, gates, None, grad_x, grad_g, buf.dev_status)
    sent = buf.send_buf.view(torch.bfloat16)
    assert (grad_x.double() * x.double()).sum() == (rows[:n].double() * sent[:n].double()).sum()
    w_sent = buf.slot_w if ll else buf.slot_local_w
    assert (grad_g.double() * w.double()).sum() == (gates[:n].double() * w_sent[:n].double()).sum()
    assert int(buf.dev_status) == 0


@pytest.mark.parametrize("ll", [False, True])
def test_rows_beyond_the_buffers(ep, ll):
    """Slots from `rows` on are reported and skipped; nothing behind is touched."""
    T, H, E, R, k = 24, 128, 16, 4, 4
    d = make(T, H, E, R, k, ll, seed=5, dropped=0.0)
    short = d["n"] - 5
    s = ep.shape(T, H, E, R, k)
    y, grad_out = d["f"](d["n"], H).bfloat16(), d["f"](T, H).bfloat16()
    grad_y = torch.full((d["n"], H), 5.0, dtype=torch.bfloat16, device="cuda")
    grad_w = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
    call(s, y[:short], d["idx"], d["w"], d["slot"], grad_out, grad_y[:short], grad_w, st)
    assert int(st) == ep.EP_ERR_CAPACITY
    assert (grad_y[short:] == 5.0).all() and not torch.isnan(grad_w).any()
    gone = [(t, j) for t, s_, js in X.served(T, E, R, k, d["idx"], d["slot"], ll) if s_ >= short for j in js]
    assert gone and all(float(grad_w[t, j]) == 0.0 for t, j in gone)
    st.zero_()
    grad_x = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    call = ep.ep_dispatch_ll_backward if ll else ep.ep_dispatch_backward
    call(s, d["idx"], d["slot"], y[:short], None, None, grad_x, None, st)
    assert int(st) == ep.EP_ERR_CAPACITY and not torch.isnan(grad_x).any()


@pytest.mark.parametrize("ll", [False, True])
def test_nothing_to_do(ep, ll):
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, **i32)
    com = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
    dis = ep.ep_dispatch_ll_backward if ll else ep.ep_dispatch_backward
    s = ep.shape(0, 64, 8, 4, 2)
    e = lambda *sh: torch.empty(*sh, **bf)  # noqa: E731
    com(s, e(5, 64), torch.empty(0, 2, **i32), torch.empty(0, 2, device="cuda"), torch.empty(0, 2 if ll else 4, **i32), e(0, 64),
        e(5, 64), torch.empty(0, 2, device="cuda"), st)
    # every choice dropped, and buffers without a row
    T = 7
    s = ep.shape(T, 64, 8, 4, 2)
    idx, slot = torch.full((T, 2), -1, **i32), torch.full((T, 2 if ll else 4), -1, **i32)
    w, grad_w = torch.ones(T, 2, device="cuda"), torch.full((T, 2), float("nan"), device="cuda")
    com(s, e(0, 64), idx, w, slot, torch.ones(T, 64, **bf), e(0, 64), grad_w, st)
    assert (grad_w == 0).all()
    grad_w.fill_(float("nan"))
    grad_x = torch.full((T, 64), float("nan"), **bf)
    dis(s, idx, slot, e(0, 64), torch.empty(0, device="cuda") if ll else torch.empty(0, 2, device="cuda"), None, grad_x, grad_w, st)
    assert (grad_x == 0).all() and (grad_w == 0).all() and int(st) == 0


def test_bad_expert_ids_are_dropped_choices(ep):
    T, H, E, R, k = 6, 64, 8, 4, 2
    idx = torch.tensor([[0, 9], [8, 1], [-1, 2], [-5, 3], [4, 2 ** 31 - 1], [-2 ** 31, 5]], dtype=torch.int32, device="cuda")
    clean = torch.where((idx < 0) | (idx >= E), -1, idx)
    f = torch.Generator(device="cuda").manual_seed(0)
    w = torch.rand(T, k, device="cuda", generator=f)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ll in (False, True):
        slot, n = X.rows_of(T, E, R, k, clean, ll)
        y = torch.randn(n, H, device="cuda", generator=f).bfloat16()
        go = torch.randn(T, H, device="cuda", generator=f).bfloat16()
        got = []
        for i in (idx, clean):
            gy, gw = torch.zeros_like(y), torch.full((T, k), float("nan"), device="cuda")
            call = ep.ep_combine_ll_backward if ll else ep.ep_combine_backward
            # a bad choice may hold any slot: it is not looked at
            at = slot.cuda() if not ll else torch.where(clean < 0, 10 ** 6, slot.cuda()).int()
            call(ep.shape(T, H, E, R, k), y, i, w, at, go, gy, gw, st)
            got.append((gy, gw))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and int(st) == 0
        assert (got[0][1][clean < 0] == 0).all()


def test_far_rows(ep):
    """Rows whose bytes lie beyond 2^32."""
    T, H, E, R, k = 3, 8192, 4, 2, 2
    cap = 300_000                       # 4.9 GB
    idx = torch.tensor([[0, 2], [1, 3], [2, 0]], dtype=torch.int32, device="cuda")
    slot = torch.tensor([[1, 299_999], [270_000, 5], [290_001, 299_998]], dtype=torch.int32, device="cuda")
    f = torch.Generator(device="cuda").manual_seed(0)
    y = torch.zeros(cap, H, dtype=torch.bfloat16, device="cuda")
    for s in slot.view(-1).tolist():
        y[s] = torch.randn(H, device="cuda", generator=f).bfloat16()
    go = torch.randn(T, H, device="cuda", generator=f).bfloat16()
    w = torch.rand(T, k, device="cuda", generator=f)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gw, gx = torch.empty(T, k, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ep.ep_dispatch_ll_backward(ep.shape(T, H, E, R, k), idx, slot, y, None, None, gx, None, st)
    at = y[slot.view(-1).long()].view(T, k, H).double()
    want = at.sum(1)
    assert_close(gx, want, X.bf16_tol(want, at.abs().sum(1) * 3 * X.U32), "grad_x")
    want = (at * go.double()[:, None]).sum(2)
    ep.ep_combine_ll_backward(ep.shape(T, H, E, R, k), y, idx, w, slot, go, y, gw, st)
    assert_close(gw, want, (at * go.double()[:, None]).abs().sum(2) * 28 * X.U32, "grad_w")
    want = w.double()[:, :, None] * go.double()[:, None]
    assert_close(y[slot.view(-1).long()].view(T, k, H), want, X.bf16_tol(want, want.abs() * 2 * X.U32), "grad_y")
    assert int(st) == 0


def test_refusals(ep):
    T, H, E, R, k = 4, 64, 8, 4, 2
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    s = ep.shape(T, H, E, R, k)
    idx, slot, w = torch.zeros(T, k, **i32), torch.zeros(T, R, **i32), torch.zeros(T, k, device="cuda")
    y, go, st = torch.zeros(9, H, **bf), torch.zeros(T, H, **bf), torch.zeros(1, **i32)
    good = dict(y=y, topk_idx=idx, topk_w=w, send_slot=slot, grad_out=go, grad_y=y.clone(), grad_topk_w=w.clone(), dev_status=st)
    bad = [dict(y=None), dict(y=y.float()), dict(y=y[:, :32]), dict(y=torch.zeros(8, H, **bf)), dict(topk_idx=idx.long()),
           dict(topk_idx=idx[:2]), dict(topk_w=None), dict(topk_w=w.double()), dict(send_slot=slot[:, :2]), dict(send_slot=None),
           dict(grad_out=None), dict(grad_out=go.float()), dict(grad_out=go[:3]), dict(grad_y=None, grad_topk_w=None),
           dict(grad_y=torch.zeros(9, 2 * H, **bf)[:, ::2]), dict(grad_topk_w=w[:1]), dict(dev_status=None), dict(y=y.cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            ep.ep_combine_backward(s, **{**good, **b})
    gates = torch.zeros(9, k, device="cuda")
    good = dict(topk_idx=idx, send_slot=slot, grad_rows=y, grad_slot_local_w=gates, grad_other=go, grad_x=go.clone(),
                grad_topk_w=w.clone(), dev_status=st)
    bad = [dict(grad_rows=None), dict(grad_rows=y[0]), dict(grad_rows=y.half()), dict(grad_slot_local_w=None), dict(grad_topk_w=None),
           dict(grad_slot_local_w=gates[:3]), dict(grad_slot_local_w=gates[:, 0]), dict(grad_other=go[:1]), dict(grad_x=None),
           dict(grad_x=go.float()), dict(dev_status=torch.zeros(2, **i32)), dict(topk_idx=None)]
    for b in bad:
        with pytest.raises(ValueError):
            ep.ep_dispatch_backward(s, **{**good, **b})
    ep.ep_dispatch_backward(s, **good)
    with pytest.raises(ep.EpError):
        ep.ep_dispatch_backward(ep.shape(T, H, E, 3, k), **{**good, "send_slot": torch.zeros(T, 3, **i32)})
