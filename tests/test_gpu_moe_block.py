"""The whole block as a user runs it: norm, router, dispatch, the experts' two
products and combine, against 64 bits with the same 8-bit roundings.

The output's norm may be off by the roundings of y and of the combined rows
(2^-8 each) and by codes near a border that fall to its other side: one in a
thousand at most by the float sums' errors, each by 2^-3 of itself, 0.4 %; in
all less than 2^-6."""

import pytest
import torch

import operator_refs as R
from gpu_helpers import log

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def make(T, H, E, F, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    w1, s1, w1_64 = R.make_weights(E, 2 * F, H, gen)
    w2, s2, w2_64 = R.make_weights(E, H, F, gen)
    return dict(x=f(T, H).bfloat16(), residual=(2 * f(T, H)).bfloat16(), weight=1 + 0.1 * f(H),
                router=f(E, H) * H ** -0.5, w1=w1, s1=s1, w2=w2, s2=s2, w1_64=w1_64, w2_64=w2_64)


def reference(d, idx, w):
    """The block in 64 bits for the given choices; zero for a token without."""
    r, _, y = R.norm64(d["x"], d["residual"], d["weight"], EPS)
    codes, scales = R.quantise(y.bfloat16().double())
    x8 = codes * scales.repeat_interleave(128, 1)
    out = torch.zeros_like(x8)
    F = d["w2_64"].shape[2]
    for e in range(d["w1_64"].shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            g = x8[t] @ d["w1_64"][e].t().contiguous()
            codes, scales = R.quantise(torch.nn.functional.silu(g[:, :F]) * g[:, F:])
            h = codes * scales.repeat_interleave(128, 1)
            out.index_add_(0, t, w[t, j].double()[:, None] * (h @ d["w2_64"][e].t().contiguous()))
    return r, out


@pytest.mark.parametrize("T,H,E,R_,k,F,masked", [(1, 256, 8, 2, 2, 128, False), (7, 512, 16, 4, 4, 256, False),
                                                 (128, 512, 16, 4, 2, 384, True), (700, 1024, 32, 8, 4, 512, True)])
def test_block(ep, T, H, E, R_, k, F, masked):
    d = make(T, H, E, F, 1)
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.uint8, device="cuda")
        mask[::5] = 0
    buf = ep.BuffersMoE(ep.shape(T, H, E, R_, k, ep.EP_FMT_FP8_E4M3_B128), F)
    log(f"[block] T={T} H={H} E={E} k={k} F={F}")
    out = buf.block(d["x"], d["residual"], d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["s1"],
                    d["w2"], d["s2"], token_mask=mask)
    assert int(buf.dev_status) == 0
    r, want = reference(d, buf.topk_idx, buf.topk_w)
    assert torch.equal(buf.residual, r)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask != 0
    idx, w, *_ = R.route64(buf.normed.float() @ d["router"].t(), keep, k, 1)
    assert torch.equal(buf.topk_idx, idx)
    assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -6
    if masked:
        assert (out[~keep] == 0).all()


def test_rows_of_the_norm_go_through_the_dispatch_as_bytes(ep):
    """The norm's 8-bit rows dispatched as opaque rows (bf16 rows of half their
    bytes) arrive at the experts byte for byte; the dense product (one group)
    takes them as they are."""
    T, H, E, k, F = 50, 512, 16, 4, 256
    d = make(T, H, E, F, 2)
    rb = R.row_bytes(H)
    rows = torch.empty(T, rb, dtype=torch.uint8, device="cuda")
    ep.ep_rmsnorm(d["x"], d["residual"], d["weight"], EPS, None, None, rows, None)
    logits = torch.randn(T, E, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ep.ep_route(logits, None, ep.EP_GATE_SOFTMAX_RENORM, idx, w)
    buf = ep.BuffersLL(ep.shape(T, rb // 2, E, 4, k))
    buf.layout(idx)
    buf.dispatch(rows.view(torch.bfloat16), idx, w)
    assert int(buf.dev_status) == 0
    assert torch.equal(buf.send_buf, rows[buf.slot_src.long()])
    y = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    inner = torch.empty(T * k, R.row_bytes(F), dtype=torch.uint8, device="cuda")
    ep.ep_expert_gate_up(buf.send_buf, buf.expert_offset, d["w1"], d["s1"], inner, buf.dev_status)
    ep.ep_expert_product(inner, buf.expert_offset, d["w2"], d["s2"], y, buf.dev_status)
    codes, scales, _ = R.split_rows(rows, H)
    x8 = (codes * scales.repeat_interleave(128, 1))[buf.slot_src.long()]
    off = buf.expert_offset.tolist()
    g = R.grouped64(x8, off, d["w1_64"])
    codes, scales = R.quantise(torch.nn.functional.silu(g[:, :F]) * g[:, F:])
    want = R.grouped64(codes * scales.repeat_interleave(128, 1), off, d["w2_64"])
    assert int(buf.dev_status) == 0
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -6
    # one group: every token through expert 0's first product
    dense = torch.empty(T, 2 * F, dtype=torch.bfloat16, device="cuda")
    ep.ep_expert_product(rows, torch.tensor([0, T], dtype=torch.int32, device="cuda"), d["w1"][:1], d["s1"][:1],
                         dense, buf.dev_status)
    x8 = R.split_rows(rows, H)
    want = (x8[0] * x8[1].repeat_interleave(128, 1)) @ d["w1_64"][0].t().contiguous()
    assert float((dense.double() - want).norm() / want.norm()) <= R.U_BF16 + 2.0 ** -13


def test_one_rank_of_the_layout(ep):
    """A rank's experts alone: its slice of expert_offset and its weights."""
    T, H, E, Rk, k, N = 300, 256, 16, 4, 4, 136
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=gen)
    w, s, w64 = R.make_weights(E, N, H, gen)
    buf = ep.BuffersLL(ep.shape(T, H, E, Rk, k, ep.EP_FMT_FP8_E4M3_B128))
    idx, gate = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ep.ep_route(logits, None, ep.EP_GATE_SOFTMAX_RENORM, idx, gate)
    buf.layout(idx)
    buf.dispatch(x, idx, gate)
    out = torch.full((T * k, N), -7.0, dtype=torch.bfloat16, device="cuda")
    e0, e1 = 4, 8          # rank 1
    ep.ep_expert_product(buf.send_buf, buf.expert_offset[e0:e1 + 1], w[e0:e1], s[e0:e1], out, buf.dev_status)
    assert int(buf.dev_status) == 0
    off = buf.expert_offset.tolist()
    codes, scales, _ = R.split_rows(buf.send_buf, H)
    want = R.grouped64(codes * scales.repeat_interleave(128, 1), off[e0:e1 + 1], w64[e0:e1])
    part = slice(off[e0], off[e1])
    assert float((out[part].double() - want[part]).norm() / want[part].norm()) <= R.U_BF16 + 2.0 ** -13
    assert (out[:off[e0]] == -7).all() and (out[off[e1]:] == -7).all()


def test_two_steps_at_once_on_two_streams(ep):
    """Two batches through the block on two streams with buffers of their own:
    each as it is alone."""
    T, H, E, k, F = 96, 512, 16, 4, 256
    sets, want = [], []
    for seed in (4, 5):
        d = make(T, H, E, F, seed)
        buf = ep.BuffersMoE(ep.shape(T, H, E, 4, k, ep.EP_FMT_FP8_E4M3_B128), F)
        run = lambda b, d: b.block(d["x"], d["residual"], d["weight"], EPS,  # noqa: E731
                                   lambda n: n.float() @ d["router"].t(), d["w1"], d["s1"], d["w2"], d["s2"])
        want.append(run(buf, d).clone())
        sets.append((buf, d, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for buf, d, s in sets:
            buf.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for buf, d, s in sets:
            with torch.cuda.stream(s):
                run(buf, d)
        torch.cuda.synchronize()
        for (buf, _, _), w in zip(sets, want):
            assert torch.equal(buf.out, w)


@pytest.mark.parametrize("T", [0, 1, 130])
def test_block_without_a_residual(ep, T):
    """A first layer has no residual: the residual stream begins as x."""
    H, E, k, F = 512, 16, 4, 256
    d = make(T, H, E, F, 6)
    d["residual"] = None
    buf = ep.BuffersMoE(ep.shape(T, H, E, 4, k, ep.EP_FMT_FP8_E4M3_B128), F)
    buf.residual.fill_(-7.0)
    out = buf.block(d["x"], None, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["s1"], d["w2"],
                    d["s2"])
    assert int(buf.dev_status) == 0
    assert out.shape == (T, H) and torch.equal(buf.residual, d["x"])
    if T:
        _, want = reference(d, buf.topk_idx, buf.topk_w)
        assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -6
    # the residual stream itself as x, as where the caller has put it there
    again = out.clone()
    assert torch.equal(buf.block(buf.residual, None, d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"],
                                 d["s1"], d["w2"], d["s2"]), again)
    assert torch.equal(buf.residual, d["x"])
    with pytest.raises(ValueError, match="x must"):      # and nothing is copied from a refused x
        buf.norm(d["x"].float(), None, d["weight"], EPS)
    assert torch.equal(buf.residual, d["x"])


@pytest.mark.parametrize("with_residual", [False, True])
def test_block_in_a_graph_and_on_a_stream(ep, with_residual):
    T, H, E, k, F = 96, 512, 16, 4, 256
    d = make(T, H, E, F, 7)
    residual = d["residual"] if with_residual else None
    buf = ep.BuffersMoE(ep.shape(T, H, E, 4, k, ep.EP_FMT_FP8_E4M3_B128), F)
    run = lambda: buf.block(d["x"], residual, d["weight"], EPS, lambda n: n.float() @ d["router"].t(),  # noqa: E731
                            d["w1"], d["s1"], d["w2"], d["s2"])
    run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    for seed in range(3):
        d["x"].copy_(make(T, H, E, F, 20 + seed)["x"])
        run()
        torch.cuda.synchronize()
        out, r = buf.out.clone(), buf.residual.clone()
        buf.out.fill_(float("nan"))
        buf.residual.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, out) and torch.equal(buf.residual, r)
    # the norm on a stream that is not the current one
    buf.residual.fill_(float("nan"))
    buf.normed.fill_(float("nan"))
    torch.cuda.synchronize()
    buf.norm(d["x"], residual, d["weight"], EPS, stream=s)
    s.synchronize()
    assert torch.equal(buf.residual, r) and torch.isfinite(buf.normed).all()


def test_block_of_padded_tokens_alone(ep):
    """No expert has a row: the output is zero, the residual stream goes on."""
    T, H, E, k, F = 20, 256, 8, 2, 128
    d = make(T, H, E, F, 8)
    buf = ep.BuffersMoE(ep.shape(T, H, E, 2, k, ep.EP_FMT_FP8_E4M3_B128), F)
    out = buf.block(d["x"], d["residual"], d["weight"], EPS, lambda n: n.float() @ d["router"].t(), d["w1"], d["s1"],
                    d["w2"], d["s2"], token_mask=torch.zeros(T, dtype=torch.uint8, device="cuda"))
    assert int(buf.dev_status) == 0 and int(buf.expert_offset.abs().max()) == 0
    assert (out == 0).all()
    assert torch.equal(buf.residual, R.norm64(d["x"], d["residual"], d["weight"], EPS)[0])


def test_an_input_of_autograd(ep):
    """x may be a tensor that autograd follows: the buffers take no part in it."""
    T, H, E, k, F = 20, 256, 8, 2, 128
    d = make(T, H, E, F, 9)
    buf = ep.BuffersMoE(ep.shape(T, H, E, 2, k, ep.EP_FMT_FP8_E4M3_B128), F)
    x = d["x"].clone().requires_grad_(True)
    side = torch.cuda.Stream()
    for stream in (None, side):
        buf.norm(x, None, d["weight"], EPS, stream=stream)
        assert not buf.residual.requires_grad and buf.residual.grad_fn is None
        torch.cuda.synchronize()
        assert torch.equal(buf.residual, d["x"])
