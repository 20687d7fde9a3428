"""The norm, router and expert-product calls without a GPU: every refusal is a
host-side check that launches nothing (the addresses here are not real)."""

import ctypes

import pytest

INVALID = 1
A = 4096            # an aligned address that is never followed


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def norm(L, T=4, H=256, x=A, residual=A, weight=A, eps=1e-6, residual_out=A, y=A, rows=A, rstd=A):
    return L.ep_rmsnorm(T, H, x, residual, weight, eps, residual_out, y, rows, rstd, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=4), dict(H=12), dict(H=32776), dict(H=-8),
    dict(H=264),                                  # 8-bit rows need whole blocks
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(weight=None), dict(y=None, rows=None), dict(residual=None),
    dict(x=A + 8), dict(residual=A + 2), dict(weight=A + 4), dict(residual_out=A + 8), dict(y=A + 8),
    dict(rows=A + 8), dict(rstd=A + 2)])
def test_norm_refuses(ep, bad):
    assert norm(ep.lib, **bad) == INVALID


def test_norm_without_rows_of_its_own(ep):
    assert norm(ep.lib, T=0) == 0
    assert norm(ep.lib, T=0, x=None, y=None, rows=None) == 0
    assert norm(ep.lib, H=40000) == INVALID
    assert b"32768" in ep.lib.ep_last_error()


def norm_back(L, T=4, H=256, r=A, weight=A, rstd=A, gy=A, gr=A, gx=A, gw=A, ws=A, n=1 << 20):
    return L.ep_rmsnorm_backward(T, H, r, weight, rstd, gy, gr, gx, gw, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=12), dict(H=32776), dict(r=None), dict(weight=None), dict(rstd=None),
    dict(gy=None), dict(gx=None), dict(gw=None), dict(ws=None), dict(n=4 * 256 * 4 - 1), dict(r=A + 8),
    dict(gy=A + 8), dict(gr=A + 8), dict(gx=A + 8), dict(gw=A + 4), dict(ws=A + 4), dict(rstd=A + 1)])
def test_norm_backward_refuses(ep, bad):
    assert norm_back(ep.lib, **bad) == INVALID


def test_workspaces(ep):
    assert ep.ep_rmsnorm_workspace_bytes(4, 256) == 4 * 256 * 4
    assert ep.ep_rmsnorm_workspace_bytes(0, 256) == 0
    assert ep.ep_rmsnorm_workspace_bytes(1 << 20, 7168) < 1 << 25
    assert ep.ep_rmsnorm_workspace_bytes(4, 12) == 0
    assert ep.ep_route_workspace_bytes(0, 8) > 0
    assert ep.ep_route_workspace_bytes(1 << 20, 4096) < 1 << 24
    assert ep.ep_route_workspace_bytes(4, 0) == 0
    assert ep.ep_route_workspace_bytes(4, 4097) == 0
    assert ep.ep_route_workspace_bytes(-1, 8) == 0


def route(L, T=4, E=16, k=2, dtype=1, mode=1, logits=A, mask=A, idx=A, w=A, counts=A, kept=A, lse=A,
          loss=A, ws=A, n=1 << 20):
    return L.ep_route(T, E, k, dtype, mode, logits, mask, idx, w, counts, kept, lse, loss, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=4097), dict(k=0), dict(k=17), dict(E=64, k=33), dict(T=1 << 30, k=2),
    dict(dtype=2), dict(dtype=-1), dict(mode=2), dict(mode=-1), dict(logits=None), dict(idx=None),
    dict(w=None), dict(counts=None), dict(kept=None), dict(loss=None), dict(ws=None), dict(n=64),
    dict(logits=A + 2), dict(dtype=0, logits=A + 1), dict(idx=A + 2), dict(w=A + 1), dict(lse=A + 2),
    dict(ws=A + 8), dict(counts=A + 2), dict(kept=A + 2), dict(loss=A + 2)])
def test_route_refuses(ep, bad):
    assert route(ep.lib, **bad) == INVALID


def test_route_of_no_tokens(ep):
    # without counts nothing is launched
    assert route(ep.lib, T=0, logits=None, idx=None, w=None, counts=None, kept=None, loss=None, ws=None,
                 n=0) == 0


def route_back(L, T=4, E=16, k=2, dtype=1, mode=1, logits=A, mask=A, idx=A, w=A, counts=A, kept=A,
               lse=A, gw=A, gl=A, out=A):
    return L.ep_route_backward(T, E, k, dtype, mode, logits, mask, idx, w, counts, kept, lse, gw, gl, out,
                               None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=4097), dict(k=17), dict(dtype=2), dict(mode=2), dict(logits=None),
    dict(idx=None), dict(w=None), dict(counts=None), dict(kept=None), dict(lse=None), dict(out=None),
    dict(logits=A + 2), dict(out=A + 2), dict(dtype=0, out=A + 1), dict(lse=A + 1), dict(gw=A + 2),
    dict(gl=A + 1), dict(idx=A + 2)])
def test_route_backward_refuses(ep, bad):
    assert route_back(ep.lib, **bad) == INVALID


def test_route_backward_of_no_tokens(ep):
    assert route_back(ep.lib, T=0, logits=None, lse=None, out=None) == 0


def product(L, G=2, M=4, N=64, K=128, rows=A, off=A, w=A, ws=A, out=A, st=A):
    return L.ep_expert_product(G, M, N, K, rows, off, w, ws, out, st, None)


def gate_up(L, G=2, M=4, F=128, K=128, rows=A, off=A, w=A, ws=A, out=A, st=A):
    return L.ep_expert_gate_up(G, M, F, K, rows, off, w, ws, out, st, None)


COMMON = [dict(G=0), dict(G=4097), dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=64), dict(K=192),
          dict(K=(1 << 20) + 128), dict(rows=None), dict(off=None), dict(w=None), dict(ws=None),
          dict(out=None), dict(st=None), dict(rows=A + 8), dict(w=A + 8), dict(out=A + 8),
          dict(off=A + 2), dict(ws=A + 2), dict(st=A + 1)]


@pytest.mark.parametrize("bad", COMMON + [dict(N=0), dict(N=4), dict(N=12), dict(N=(1 << 24) + 8)])
def test_product_refuses(ep, bad):
    assert product(ep.lib, **bad) == INVALID


@pytest.mark.parametrize("bad", COMMON + [dict(F=0), dict(F=64), dict(F=192), dict(F=1 << 24)])
def test_gate_up_refuses(ep, bad):
    assert gate_up(ep.lib, **bad) == INVALID


def test_products_of_no_rows(ep):
    assert product(ep.lib, M=0, rows=None, out=None) == 0
    assert gate_up(ep.lib, M=0, rows=None, out=None) == 0


def test_too_many_tiles_is_refused(ep):
    assert product(ep.lib, G=4096, M=(1 << 31) - 1, N=1 << 24, K=128) == INVALID
    assert b"tiles" in ep.lib.ep_last_error()


def test_row_bytes_of_the_binding(ep):
    for H in [128 * i for i in range(1, 200)] + [1 << 20]:
        assert ep._row8(H) == ep.ep_row_bytes(H, ep.EP_FMT_FP8_E4M3_B128)


def test_python_names_a_wrong_tensor(ep):
    """The binding's own checks, on tensors of the CPU: the current device is
    taken as theirs (-1)."""
    import torch
    ep._types()
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    assert ep._arg("x", None, torch.bfloat16, (4, 256), -1) is None
    assert ep._arg("x", t, torch.bfloat16, (4, 256), -1) == t.data_ptr()
    for args in [(t, torch.float32, (4, 256), -1), (t, torch.bfloat16, (4, 128), -1),
                 (t[:, ::2], torch.bfloat16, (4, 128), -1), (t, torch.bfloat16, (4, 256), 0)]:
        with pytest.raises(ValueError, match="x must"):
            ep._arg("x", *args)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ep._logits_type(torch.zeros(2, 2, dtype=torch.float64))
    with pytest.raises(ValueError):
        ep.BuffersMoE(ep.shape(4, 256, 8, 2, 2), 128, device="cpu")
    assert isinstance(ep.lib, ctypes.CDLL)
