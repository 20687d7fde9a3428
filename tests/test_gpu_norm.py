"""ep_rmsnorm and its backward against 64 bits.

Tolerances: a thread adds up to 32 squares in a row, then six steps in the
wavefront and up to 16 wavefronts: the sum of squares is off by 56 roundings,
the root by half of that, and rstd, y = r * rstd * weight by four more: REL."""

import pytest
import torch

import operator_refs as R
from gpu_helpers import log

pytestmark = pytest.mark.gpu

REL = 40 * R.U32
EPS = 1e-5


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def make(T, H, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    spread = 1.0 + 7.0 * (torch.rand(H, device="cuda", generator=g) < 0.02)
    return ((f(T, H) * spread).bfloat16(), (2 * f(T, H) * spread).bfloat16(), 1 + 0.2 * f(H), f)


def outputs(ep, T, H, residual=True, y=True, rows=True, rstd=True):
    bf = dict(dtype=torch.bfloat16, device="cuda")
    return dict(residual_out=torch.full((T, H), float("nan"), **bf) if residual else None,
                y=torch.full((T, H), float("nan"), **bf) if y else None,
                rows=torch.full((T, R.row_bytes(H)), 0xA5, dtype=torch.uint8, device="cuda") if rows else None,
                rstd=torch.full((T,), float("nan"), device="cuda") if rstd else None)


def check(o, x, residual, weight, eps=EPS):
    r, rstd, y = R.norm64(x, residual, weight, eps)
    if o["residual_out"] is not None:
        assert torch.equal(o["residual_out"], r)
    if o["rstd"] is not None:
        R.assert_close(o["rstd"], rstd, rstd * REL, "rstd")
    if o["y"] is not None:
        R.assert_close(o["y"], y, y.abs() * (R.U_BF16 * (1 + REL) + REL) + 2.0 ** -133, "y")
    if o["rows"] is not None:
        R.assert_rows8(o["rows"], y, REL, "rows")


@pytest.mark.parametrize("T,H", [(1, 8), (3, 72), (5, 128), (33, 128), (17, 384), (2, 512), (4, 520), (9, 640),
                                 (300, 1024), (7, 4096), (1, 7168), (130, 7168), (2, 8192), (3, 8200), (2, 16384),
                                 (2, 16640), (3, 32768), (2, 32760), (5000, 256)])
def test_forward(ep, T, H):
    x, res, w, _ = make(T, H)
    log(f"[norm] T={T} H={H}")
    o = outputs(ep, T, H, rows=H % 128 == 0)
    ep.ep_rmsnorm(x, res, w, EPS, **o)
    check(o, x, res, w)


@pytest.mark.parametrize("residual,residual_out,y,rows,rstd", [
    (False, False, True, False, False), (False, False, False, True, True), (True, False, True, True, False),
    (True, True, False, True, False), (True, True, True, False, True)])
def test_optional_outputs(ep, residual, residual_out, y, rows, rstd):
    T, H = 19, 896
    x, res, w, _ = make(T, H, 1)
    o = outputs(ep, T, H, residual_out, y, rows, rstd)
    ep.ep_rmsnorm(x, res if residual else None, w, EPS, **o)
    check(o, x, res if residual else None, w)


@pytest.mark.parametrize("over", ["residual_out=x", "residual_out=residual", "y=x", "y=x, residual_out=residual"])
def test_in_place(ep, over):
    T, H = 600, 7168
    x, res, w, _ = make(T, H, 2)
    x0, res0 = x.clone(), res.clone()
    o = outputs(ep, T, H)
    for pair in over.split(", "):
        k, v = pair.split("=")
        o[k] = x if v == "x" else res
    ep.ep_rmsnorm(x, res, w, EPS, **o)
    check(o, x0, res0, w)


def test_values_that_are_not_ordinary(ep):
    """A zero row (eps alone under the root), tiny and huge rows, a NaN and an
    infinity: other rows stay clean, and so do the blocks without them."""
    T, H = 8, 512
    x, _, w, _ = make(T, H, 3)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e15
    x[3, 200] = float("nan")
    x[4, 300] = float("inf")
    o = outputs(ep, T, H, residual=False)
    ep.ep_rmsnorm(x, None, w, EPS, **o)
    good = [0, 1, 2, 5, 6, 7]
    check({k: None if v is None else v[good] for k, v in o.items()}, x[good], None, w)
    assert torch.isnan(o["y"][3]).all() and torch.isnan(o["rstd"][3])
    assert o["rstd"][4] == 0 and torch.isnan(o["y"][4, 300]) and (o["y"][4, :300] == 0).all()
    codes, scales, _ = R.split_rows(o["rows"], H)
    assert torch.isnan(codes[3]).all() and torch.isnan(codes[4, 300])
    assert (scales[3:5] == torch.tensor(1e-4 / 448, device="cuda").double()).all() or \
        torch.allclose(scales[3:5], torch.full_like(scales[3:5], 1e-4 / 448.0), rtol=1e-6)


@pytest.mark.parametrize("H", [512, 7168])
def test_limits_of_the_sum_of_squares(ep, H):
    """Rows at the ends of what the header states: up to a root mean square of
    1.8e19 / sqrt(H) they are normalised, beyond it y is 0; with eps = 0 down to
    1e-18, and below 2^-75 rstd is infinite."""
    _, _, w, f = make(5, H, 6)
    sign = torch.where(f(5, H) < 0, -1.0, 1.0)
    size = torch.tensor([1.7e19 / H ** 0.5, 1.9e19 / H ** 0.5, 1e-18, 2.0 ** -76, 1.0], device="cuda")
    x = (sign * size[:, None]).bfloat16()
    o = outputs(ep, 5, H, residual=False)
    ep.ep_rmsnorm(x, None, w, 0.0, **o)
    good = [0, 2, 4]
    check({k: None if v is None else v[good] for k, v in o.items()}, x[good], None, w, 0.0)
    assert o["rstd"][1] == 0 and (o["y"][1] == 0).all()
    assert torch.isinf(o["rstd"][3]) and torch.isinf(o["y"][3]).all()


def test_overflowing_elements_take_the_dispatch_codes(ep):
    """A weight that makes y infinite: the block's scale is infinite, its finite
    elements are zero and the infinite one is the NaN code with its sign, as
    ep_dispatch packs such rows."""
    T, H = 2, 256
    x, _, w, _ = make(T, H, 4)
    w[5] = float("inf")
    x[0, 5], x[1, 5] = 1.0, -1.0
    o = outputs(ep, T, H, residual=False, y=False)
    ep.ep_rmsnorm(x, None, w, EPS, **o)
    raw = o["rows"][:, :H]
    assert raw[0, 5] == 0x7F and raw[1, 5] == 0xFF
    _, scales, _ = R.split_rows(o["rows"], H)
    assert torch.isinf(scales[:, 0]).all() and torch.isfinite(scales[:, 1]).all()
    rest = torch.cat([raw[:, :5], raw[:, 6:128]], 1)
    assert ((rest & 0x7F) == 0).all()


def test_empty(ep):
    o = outputs(ep, 0, 256)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    ep.ep_rmsnorm(x, x, torch.ones(256, device="cuda"), EPS, **o)
    gw = torch.full((256,), 7.0, device="cuda")
    ep.ep_rmsnorm_backward(x, torch.ones(256, device="cuda"), o["rstd"], x, None, x, gw, None)
    assert (gw == 0).all()


def back(ep, x, w, rstd, gy, gr, gx=None):
    T, H = x.shape
    gx = torch.full_like(x, float("nan")) if gx is None else gx
    gw = torch.full((H,), float("nan"), device="cuda")
    ws = torch.full((ep.ep_rmsnorm_workspace_bytes(T, H),), 0xFF, dtype=torch.uint8, device="cuda")
    ep.ep_rmsnorm_backward(x, w, rstd, gy, gr, gx, gw, ws)
    return gx, gw


def check_back(gx, gw, x, w, rstd, gy, gr):
    """grad_x: bf16's rounding and 80 float roundings of its largest parts (the
    mean of g h is a sum of 32 + 6 + 16 steps over terms of three roundings);
    grad_weight: a column's sum runs over T / 512 rows a workgroup, 32
    workgroups a slice and 16 slices."""
    T = x.shape[0]
    dx, dw = R.norm_back64(x, w, rstd, gy, gr)
    h = (x.double() * rstd.double()[:, None]).abs()
    g = (gy.double() * w.double()).abs()
    parts = rstd.double()[:, None] * (g + h * (g * h).mean(1, keepdim=True))
    if gr is not None:
        parts = parts + gr.double().abs()
    R.assert_close(gx, dx, dx.abs() * R.U_BF16 + 80 * R.U32 * parts + 2.0 ** -133, "grad_x")
    n = -(-T // 512) + 32 + 16 + 4
    R.assert_close(gw, dw, n * R.U32 * (gy.double().abs() * h).sum(0), "grad_weight")


@pytest.mark.parametrize("T,H,residual", [(1, 8, False), (3, 72, True), (33, 128, True), (511, 384, False),
                                          (513, 640, True), (1100, 1024, True), (4, 7168, True), (700, 7168, False),
                                          (20, 8200, True), (6, 16640, True), (5, 32768, True), (2100, 264, True)])
def test_backward(ep, T, H, residual):
    x, _, w, f = make(T, H, 5)
    gy = f(T, H).bfloat16()
    gr = f(T, H).bfloat16() if residual else None
    _, rstd, _ = R.norm64(x, None, w, EPS)
    rstd = rstd.float()
    log(f"[norm backward] T={T} H={H}")
    check_back(*back(ep, x, w, rstd, gy, gr), x, w, rstd, gy, gr)


@pytest.mark.parametrize("over", ["grad_y", "grad_residual"])
def test_backward_in_place(ep, over):
    x, _, w, f = make(600, 1024, 6)
    gy, gr = f(600, 1024).bfloat16(), f(600, 1024).bfloat16()
    rstd = R.norm64(x, None, w, EPS)[1].float()
    gy0, gr0 = gy.clone(), gr.clone()
    gx, gw = back(ep, x, w, rstd, gy, gr, gx=gy if over == "grad_y" else gr)
    check_back(gx, gw, x, w, rstd, gy0, gr0)


def test_backward_against_differences(ep):
    """Along random directions, the loss sum(y * c) in 64 bits moves as the
    kernel's gradients say.  A central difference of step e is off by e^2 times
    the third derivative (1e-6 here); the gradients by bf16's rounding."""
    T, H, e = 3, 256, 1e-4
    x, _, w, f = make(T, H, 7)
    c = f(T, H).bfloat16()
    rstd = R.norm64(x, None, w, EPS)[1].float()
    gx, gw = back(ep, x, w, rstd, c, None)

    def loss(xd, wd):
        return (xd / torch.sqrt((xd * xd).mean(1, keepdim=True) + EPS) * wd * c.double()).sum()

    xd, wd = x.double(), w.double()
    for _ in range(4):
        u, v = f(T, H).double(), f(H).double()
        num = (loss(xd + e * u, wd) - loss(xd - e * u, wd)) / (2 * e)
        assert abs(float(num - (gx.double() * u).sum())) <= float((gx.double() * u).abs().sum()) * R.U_BF16 + 1e-5
        num = (loss(xd, wd + e * v) - loss(xd, wd - e * v)) / (2 * e)
        assert abs(float(num - (gw.double() * v).sum())) <= float((gw.double() * v).abs().sum()) * 1e-5 + 1e-5


def test_other_stream_and_graph(ep):
    T, H = 64, 1024
    x, res, w, f = make(T, H, 8)
    o = outputs(ep, T, H)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ep.ep_rmsnorm(x, res, w, EPS, **o, stream=s)
    s.synchronize()
    check(o, x, res, w)
    gy = f(T, H).bfloat16()
    gx, gw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.zeros(ep.ep_rmsnorm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ep.ep_rmsnorm(x, res, w, EPS, **o)
        ep.ep_rmsnorm_backward(o["residual_out"], w, o["rstd"], gy, None, gx, gw, ws)
    for seed in (9, 10, 11):
        x2, res2, _, f2 = make(T, H, seed)
        x.copy_(x2)
        res.copy_(res2)
        gy.copy_(f2(T, H))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        check(o, x, res, w)
        check_back(gx, gw, o["residual_out"], w, o["rstd"], gy, None)


def test_refusals_by_the_binding(ep):
    x, res, w, _ = make(4, 256)
    o = outputs(ep, 4, 256)
    for bad in [dict(x=x.float()), dict(x=x[:, ::2]), dict(x=x.cpu()), dict(x=None), dict(residual=res[:3]),
                dict(weight=w.double()), dict(weight=w[:128]), dict(weight=None), dict(y=o["y"][:, :128]),
                dict(rows=o["rows"][:, :256].contiguous()), dict(rstd=o["rstd"][:2]), dict(x=x[0])]:
        a = {**dict(x=x, residual=res, weight=w, eps=EPS, **o), **bad}
        with pytest.raises(ValueError):
            ep.ep_rmsnorm(**a)
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm(x, res, w, -1.0, **o)
    with pytest.raises(ValueError):
        ep.ep_rmsnorm_backward(x, w, o["rstd"], x, None, x, torch.empty(256, device="cuda"), None)
    with pytest.raises(ep.EpError):
        ep.ep_rmsnorm_backward(x, w, o["rstd"], x, None, x, torch.empty(256, device="cuda"),
                               torch.empty(64, device="cuda"))
