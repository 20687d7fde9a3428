"""The training pass's calls without a GPU: every refusal is a host-side check
that launches nothing (the addresses here are not real)."""

import ctypes

import pytest

INVALID = 1
A = 4096            # an aligned address that is never followed


@pytest.fixture(scope="module")
def ep():
    import combine_topk_rank_amd as ep
    return ep


def exchange(ep, name, T=4, H=64, E=8, R=4, k=2, fmt=0, **over):
    s = ep.shape(T, H, E, R, k, fmt)
    if name.startswith("ep_combine"):
        a = dict(y=A, rows=9, idx=A, w=A, slot=A, go=A, gy=A, gw=A, st=A)
    else:
        a = dict(idx=A, slot=A, gr=A, rows=9, gates=A, other=A, gx=A, gw=A, st=A)
    a.update(over)
    return getattr(ep.lib, name)(ctypes.byref(s), *a.values(), None)


COMBINE = ["ep_combine_backward", "ep_combine_ll_backward"]
DISPATCH = ["ep_dispatch_backward", "ep_dispatch_ll_backward"]


@pytest.mark.parametrize("name", COMBINE)
@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=4), dict(H=12), dict(E=9), dict(R=0), dict(R=65, E=65), dict(k=0), dict(k=9), dict(k=33, E=64),
    dict(fmt=2), dict(fmt=1), dict(y=None), dict(rows=-1), dict(idx=None), dict(w=None), dict(slot=None), dict(go=None),
    dict(gy=None, gw=None), dict(st=None), dict(y=A + 8), dict(go=A + 4), dict(gy=A + 2), dict(idx=A + 2), dict(w=A + 1),
    dict(slot=A + 2), dict(gw=A + 2), dict(st=A + 2), dict(T=1 << 30, R=4)])
def test_combine_refuses(ep, name, bad):
    assert exchange(ep, name, **bad) == INVALID


@pytest.mark.parametrize("name", DISPATCH)
@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=4), dict(H=12), dict(E=9), dict(R=0), dict(R=65, E=65), dict(k=0), dict(k=9), dict(k=33, E=64),
    dict(fmt=2), dict(gr=None), dict(rows=-1), dict(idx=None), dict(slot=None), dict(gates=None), dict(gw=None), dict(gx=None),
    dict(st=None), dict(gr=A + 8), dict(other=A + 4), dict(gx=A + 2), dict(gates=A + 2), dict(gw=A + 1), dict(idx=A + 2),
    dict(slot=A + 2), dict(st=A + 1)])
def test_dispatch_refuses(ep, name, bad):
    assert exchange(ep, name, **bad) == INVALID


@pytest.mark.parametrize("name", COMBINE + DISPATCH)
def test_no_tokens(ep, name):
    assert exchange(ep, name, T=0) == 0
    over = dict(y=None, gy=None, gw=None) if name in COMBINE else dict(gr=None, gx=None, gates=None, gw=None, other=None)
    assert exchange(ep, name, T=0, idx=None, slot=None, **over) == 0
    assert exchange(ep, name, T=0, st=None) == INVALID


def product(L, G=2, M=9, N=64, K=72, rows=A, off=A, w=A, out=A, st=A):
    return L.ep_expert_product_bf16(G, M, N, K, rows, off, w, out, st, None)


def gate(L, G=2, M=9, F=32, K=72, rows=A, off=A, w=A, pre=A, out=A, st=A):
    return L.ep_expert_gate_up_bf16(G, M, F, K, rows, off, w, pre, out, st, None)


SHARED = [dict(G=0), dict(G=4097), dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=4), dict(K=76), dict(K=(1 << 20) + 8), dict(K=-8),
          dict(rows=None), dict(off=None), dict(w=None), dict(st=None), dict(rows=A + 8), dict(w=A + 8), dict(off=A + 2),
          dict(st=A + 2)]
FORWARD = SHARED + [dict(out=None), dict(out=A + 8)]


@pytest.mark.parametrize("bad", FORWARD + [dict(N=0), dict(N=12), dict(N=(1 << 20) + 8)])
def test_product_refuses(ep, bad):
    assert product(ep.lib, **bad) == INVALID


@pytest.mark.parametrize("bad", FORWARD + [dict(F=0), dict(F=12), dict(F=(1 << 19) + 8), dict(F=-8), dict(F=1 << 30), dict(pre=A + 8)])
def test_gate_refuses(ep, bad):
    assert gate(ep.lib, **bad) == INVALID


def test_no_rows_launch_nothing(ep):
    assert product(ep.lib, M=0) == 0 and product(ep.lib, M=0, rows=None, out=None) == 0
    assert gate(ep.lib, M=0) == 0 and gate(ep.lib, M=0, rows=None, out=None, pre=None) == 0
    assert product_back(ep.lib, M=0, gw=None) == 0
    assert gate_back(ep.lib, M=0, gw=None) == 0
    assert product(ep.lib, M=0, N=12) == INVALID


def product_back(L, G=2, M=9, N=64, K=72, dtype=0, rows=A, off=A, w=A, go=A, gr=A, gw=A, st=A, ws=A, n=1 << 30):
    return L.ep_expert_product_bf16_backward(G, M, N, K, dtype, rows, off, w, go, gr, gw, st, ws, n, None)


def gate_back(L, G=2, M=9, F=32, K=72, dtype=0, rows=A, off=A, w=A, pre=A, go=A, gp=A, gr=A, gw=A, st=A, ws=A, n=1 << 30):
    return L.ep_expert_gate_up_bf16_backward(G, M, F, K, dtype, rows, off, w, pre, go, gp, gr, gw, st, ws, n, None)


BACK = SHARED + [dict(dtype=2), dict(dtype=-1), dict(go=None), dict(go=A + 8), dict(gr=A + 8), dict(gw=A + 4),
                 dict(G=1, M=100_000, ws=None), dict(G=1, M=100_000, n=64), dict(G=1, M=100_000, ws=A + 8)]


@pytest.mark.parametrize("bad", BACK + [dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(gr=None, gw=None)])
def test_product_backward_refuses(ep, bad):
    assert product_back(ep.lib, **bad) == INVALID


@pytest.mark.parametrize("bad", BACK + [dict(F=0), dict(F=12), dict(F=(1 << 19) + 8), dict(pre=None), dict(pre=A + 8), dict(gp=None),
                                        dict(gp=A + 8)])
def test_gate_backward_refuses(ep, bad):
    assert gate_back(ep.lib, **bad) == INVALID


def test_workspaces(ep):
    need = ep.ep_expert_backward_workspace_bytes
    assert need(8, 8192, 7168, 1792) == 0          # tiles enough without parts
    assert need(1, 100, 64, 64) == 0               # one block of rows
    assert 0 < need(1, 100_000, 64, 64) < 1 << 26
    for bad in ((0, 8, 64, 64), (1, -1, 64, 64), (1, 8, 12, 64), (1, 8, 64, 4), (4097, 8, 64, 64), (1, 1 << 31, 64, 64)):
        assert need(*bad) == 0
    assert all(need(G, M, N, K) < 1 << 30 for G in (1, 7, 4096) for M in (0, 1, 10 ** 6, 2 ** 31 - 1) for N in (8, 4096) for K in (8, 4096))
    assert 0 < ep.ep_grad_norm_workspace_bytes() < 1 << 16


def table(ep, *tensors, buffer=True, into=True):
    """ep_tensor_table's status, the list and the bytes of the table."""
    n = len(tensors)
    a = (ep.ep_tensor_t * max(1, n))(*[ep.ep_tensor_t(*x) for x in tensors])
    out, lst = ctypes.create_string_buffer(ep.lib.ep_tensor_table_bytes(n)), ep.ep_tensor_list_t()
    st = ep.lib.ep_tensor_table(n, a, out if buffer else None, ctypes.byref(lst) if into else None)
    return st, lst, out.raw


@pytest.mark.parametrize("bad", [(A, -1, 0, 0), (A, 1 << 38, 0, 0), (A, 4, 2, 0), (A, 4, -1, 0), (None, 4, 0, 0), (A + 1, 4, 0, 0),
                                 (A + 2, 4, 1, 0)])
def test_a_bad_tensor(ep, bad):
    assert table(ep, bad)[0] == INVALID
    assert table(ep, (A, 8, 1, 0), bad)[0] == INVALID


def test_table(ep):
    assert ep.lib.ep_tensor_table_bytes(-1) == 0
    assert table(ep, buffer=False)[0] == INVALID and table(ep, into=False)[0] == INVALID
    st, lst, _ = table(ep)
    assert st == 0 and lst.count == 0 and lst.units == 0
    # a unit is 16384 elements from the first 128-byte boundary on; what lies before is the first's
    sizes = [(A, 1, 1), (A + 4, 31, 1), (A + 4, 32, 1), (A, 0, 0), (A + 2, 16384 + 63, 0), (A + 2, 16384 + 64, 0), (None, 0, 1), (A, 1 << 30, 0)]
    st, lst, raw = table(ep, *[(*x, 0) for x in sizes])
    assert st == 0 and lst.count == 8
    import struct
    entries = [struct.unpack_from("<QqI", raw, 32 * i) for i in range(8)]
    assert [e[2] for e in entries] == [0, 1, 2, 3, 3, 4, 6, 6]
    assert struct.unpack_from("<I", raw, 32 * 8 + 16)[0] == lst.units == 6 + (1 << 16)
    assert [e[0] for e in entries] == [(x[0] or 0) | x[2] for x in sizes] and [e[1] for e in entries] == [x[1] for x in sizes]
    # too many units
    assert table(ep, *[(A, (1 << 38) - 1, 0, 0)] * 129)[0] == INVALID
    assert b"2^31" in ep.lib.ep_last_error()


def listed(ep, *sizes, at=A):
    lst = table(ep, *[(A, n, 0, 0) for n in sizes])[1]
    lst.table = at
    return lst


def norm(ep, lst, s=A, n=A, ws=A, bytes_=1 << 20):
    return ep.lib.ep_grad_norm(ctypes.byref(lst) if lst else None, s, n, ws, bytes_, None)


def clip(ep, lst, into=None, s=A, bound=1.0):
    return ep.lib.ep_grad_clip(ctypes.byref(lst) if lst else None, ctypes.byref(into) if into else None, s, bound, None)


def test_lists_that_are_none(ep):
    for lst in (None, listed(ep, 8, at=None), listed(ep, 8, at=A + 8)):
        assert norm(ep, lst) == INVALID
        assert clip(ep, lst) == INVALID
        if lst is not None:
            assert clip(ep, listed(ep, 8), lst) == INVALID
    lst = listed(ep, 8)
    lst.units = -1
    assert norm(ep, lst) == INVALID and clip(ep, lst) == INVALID
    lst.units = 1 << 31
    assert norm(ep, lst) == INVALID


def test_norm_refuses(ep):
    lst = listed(ep, 8)
    for bad in (dict(s=None), dict(s=A + 4), dict(n=A + 2), dict(ws=None), dict(ws=A + 8), dict(bytes_=64)):
        assert norm(ep, lst, **bad) == INVALID, bad


def test_clip_refuses(ep):
    lst = listed(ep, 8, 9)
    for bad in (dict(s=None), dict(s=A + 4), dict(bound=-1.0), dict(bound=float("nan")), dict(into=listed(ep, 8)),
                dict(into=listed(ep, 9, 8)), dict(into=listed(ep, 8, 10))):
        assert clip(ep, lst, **bad) == INVALID, bad
    # nothing to launch
    assert clip(ep, listed(ep, at=None)) == 0
    assert clip(ep, listed(ep, 0, 0, at=None)) == 0


def test_a_block_with_weights_gradients_of_no_such_type(ep):
    import torch
    for kind in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="weights_dtype"):
            ep.BuffersMoETrain(ep.shape(4, 64, 8, 4, 2), 32, weights_dtype=kind, device="cpu")


def test_which_tiles(ep):
    """The plan of the bf16 products: one row an expert is a weight stream through small tiles, a training batch's rows go
    through big ones; what the calls refuse is refused."""
    plan, small, big = ep.ep_expert_bf16_plan, ep.EP_TILES_SMALL, ep.EP_TILES_BIG
    for p in (ep.EP_PRODUCT_FORWARD, ep.EP_PRODUCT_GATE_UP, ep.EP_PRODUCT_ROWS_BACKWARD):
        assert plan(p, 8, 8, 7168, 1792) == small and plan(p, 8, 8192, 7168, 1792) == big
    p = ep.EP_PRODUCT_WEIGHTS_BACKWARD
    assert plan(p, 8, 8, 7168, 1792) == big and plan(p, 32, 8192, 512, 1024) == small
    assert plan(p, 1, 100_000, 64, 64) == big           # in parts
    L = ep.lib.ep_expert_bf16_plan
    for bad in ((-1, 2, 9, 64, 72), (4, 2, 9, 64, 72), (0, 0, 9, 64, 72), (0, 4097, 9, 64, 72), (0, 2, -1, 64, 72), (0, 2, 1 << 31, 64, 72),
                (0, 2, 9, 12, 72), (0, 2, 9, 64, 76), (0, 2, 9, (1 << 20) + 8, 72), (1, 2, 9, 72, 72)):
        assert L(*bad) == INVALID, bad
        with pytest.raises(ep.EpError):
            plan(*bad)
    assert all(L(p, G, M, N, K) in (small, big) for p in range(4) for G in (1, 70, 4096) for M in (0, 1, 10 ** 6, 2 ** 31 - 1)
               for N in (16, 4096, 1 << 20) for K in (8, 4096, 1 << 20))
