"""Python binding of libep.so (include/ep.h): MoE expert-parallel dispatch and
combine on one MI355X.

Argument marshalling only.  Every step of the path runs in the HIP kernels of
libep.so; torch supplies device memory and streams.  There is no fallback:
importing this package fails loudly when libep.so has not been built
(``python combine_topk_rank_amd/build.py``).

The functions keep the C names:

    ep_row_bytes(H, fmt) -> int
    ep_workspace_bytes(shape) -> int
    ep_dispatch_layout(shape, topk_idx, num_tokens_per_rank, num_tokens_per_expert,
                       rank_offset, expert_offset, is_token_in_rank, send_slot,
                       workspace, dev_status, stream=None)
    ep_dispatch(shape, x, topk_idx, topk_w, rank_offset, send_slot, send_buf,
                slot_src, slot_local_idx, slot_local_w, ring, workspace,
                dev_status, stream=None)
    ep_dispatch_fused_plan(shape, with_ring=True) -> int
    ep_dispatch_fused_noalloc(shape, x, topk_idx, topk_w, <layout outputs>, send_buf,
                              slot_src, slot_local_idx, slot_local_w, ring, dev_status,
                              stream=None, clear_scratch=False)
    ep_dispatch_ll_layout(shape, topk_idx, num_tokens_per_expert, expert_offset, expert_slot,
                          workspace, dev_status, stream=None)
    ep_combine(shape, y, topk_idx, topk_w, send_slot, out, dev_status, stream=None)
        (y_rows is y.shape[0])
    ep_rmsnorm(x, residual, weight, eps, residual_out, y, rows, rstd, stream=None)
    ep_rmsnorm_backward(r, weight, rstd, grad_y, grad_residual, grad_x, grad_weight,
                        workspace, stream=None)
    ep_route(logits, token_mask, mode, topk_idx, topk_w, num_tokens_per_expert, num_tokens,
             lse, balance_loss, workspace, stream=None)
    ep_route_backward(logits, token_mask, mode, topk_idx, topk_w, num_tokens_per_expert,
                      num_tokens, lse, grad_topk_w, grad_balance_loss, grad_logits, stream=None)
    ep_expert_product(rows, group_offset, w, w_scale, out, dev_status, stream=None)
    ep_expert_gate_up(rows, group_offset, w, w_scale, out_rows, dev_status, stream=None)
        (these six take their sizes from the tensors and check every one: a wrong type,
        shape, device or stride raises ValueError)
    Ring(depth, channels, max_inflight, timeout_ns)   # ep_ring_* calls

Tensors are torch tensors on the current HIP device (contiguous); ``stream``
defaults to torch's current stream.  A non-OK return raises EpError.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep.so")

EP_OK = 0
EP_ERR_INVALID_ARG = 1
EP_ERR_BAD_EXPERT = 2
EP_ERR_CAPACITY = 3
EP_ERR_RING_TIMEOUT = 4
EP_ERR_HIP = 5
EP_ERR_BUSY = 6
EP_ERR_TIMEOUT = 7
EP_FUSED_ONE_KERNEL_SMALL = 101
EP_FUSED_ONE_KERNEL_LARGE = 102
EP_FUSED_TWO_CALLS = 103
EP_FMT_BF16 = 0
EP_FMT_FP8_E4M3_B128 = 1
EP_BF16 = 0
EP_F32 = 1
EP_GATE_SOFTMAX = 0
EP_GATE_SOFTMAX_RENORM = 1
EP_CMD_WRITE = 1
EP_CMD_ATOMIC = 2
EP_ATOMIC_ADD = 1

# ep_transfer_cmd_t, 32 bytes
CMD_DTYPE = np.dtype([
    ("seq", "<u4"), ("type", "u1"), ("op", "u1"), ("num_tokens", "<u2"),
    ("dst_rank", "<u4"), ("size_or_value", "<u4"),
    ("src_offset", "<u8"), ("dst_offset", "<u8"),
])


class EpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status == EP_ERR_HIP:
            detail = " [" + lib.ep_last_error().decode() + "]"
        super().__init__(f"{where}: {status_str(status)} ({status}){detail}")


class ep_shape_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("R", ctypes.c_int32), ("k", ctypes.c_int32), ("fmt", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    # torch ships its own HIP runtime (file libamdhip64.so, soname
    # libamdhip64.so.7).  Loading torch first lets libep.so's dependency on
    # libamdhip64.so.7 resolve to that same runtime; the other order puts two
    # HIP runtimes in the process and the second one finds no device.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python combine_topk_rank_amd/build.py` "
                          "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    S = ctypes.POINTER(ep_shape_t)
    L.ep_row_bytes.argtypes = [i32, i32]
    L.ep_row_bytes.restype = sz
    L.ep_workspace_bytes.argtypes = [S]
    L.ep_workspace_bytes.restype = sz
    L.ep_dispatch_layout.argtypes = [S, P, P, P, P, P, P, P, P, sz, P, P]
    L.ep_dispatch_layout.restype = ctypes.c_int
    L.ep_dispatch.argtypes = [S, P, P, P, P, P, P, i64, P, P, P, P, P, sz, P, P]
    L.ep_dispatch.restype = ctypes.c_int
    L.ep_dispatch_fused.argtypes = [S, P, P, P, P, P, P, P, P, P, P, i64, P, P, P, P, P, sz, P,
                                    P]
    L.ep_dispatch_fused.restype = ctypes.c_int
    L.ep_dispatch_fused_plan.argtypes = [S, i32]
    L.ep_dispatch_fused_plan.restype = ctypes.c_int
    L.ep_dispatch_fused_noalloc.argtypes = [S, P, P, P, P, P, P, P, P, P, P, i64, P, P, P, P,
                                            i32, P, P]
    L.ep_dispatch_fused_noalloc.restype = ctypes.c_int
    L.ep_combine.argtypes = [S, P, i64, P, P, P, P, P, P]
    L.ep_combine.restype = ctypes.c_int
    L.ep_dispatch_layout_ll.argtypes = [S, P, P, P, P, sz, P, P]
    L.ep_dispatch_layout_ll.restype = ctypes.c_int
    L.ep_dispatch_ll_layout.argtypes = [S, P, P, P, P, P, sz, P, P]
    L.ep_dispatch_ll_layout.restype = ctypes.c_int
    L.ep_dispatch_ll.argtypes = [S, P, P, P, P, P, P, i64, P, P, P, P, sz, P, P]
    L.ep_dispatch_ll.restype = ctypes.c_int
    L.ep_dispatch_ll_fused.argtypes = [S, P, P, P, P, P, P, P, i64, P, P, P, P, sz, P, P]
    L.ep_dispatch_ll_fused.restype = ctypes.c_int
    L.ep_combine_ll.argtypes = [S, P, i64, P, P, P, P, P, P]
    L.ep_combine_ll.restype = ctypes.c_int
    f32 = ctypes.c_float
    L.ep_rmsnorm.argtypes = [i32, i32, P, P, P, f32, P, P, P, P, P]
    L.ep_rmsnorm.restype = ctypes.c_int
    L.ep_rmsnorm_workspace_bytes.argtypes = [i32, i32]
    L.ep_rmsnorm_workspace_bytes.restype = sz
    L.ep_rmsnorm_backward.argtypes = [i32, i32, P, P, P, P, P, P, P, P, sz, P]
    L.ep_rmsnorm_backward.restype = ctypes.c_int
    L.ep_route_workspace_bytes.argtypes = [i32, i32]
    L.ep_route_workspace_bytes.restype = sz
    L.ep_route.argtypes = [i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, sz, P]
    L.ep_route.restype = ctypes.c_int
    L.ep_route_backward.argtypes = [i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P]
    L.ep_route_backward.restype = ctypes.c_int
    L.ep_expert_product.argtypes = [i32, i64, i32, i32, P, P, P, P, P, P, P]
    L.ep_expert_product.restype = ctypes.c_int
    L.ep_expert_gate_up.argtypes = [i32, i64, i32, i32, P, P, P, P, P, P, P]
    L.ep_expert_gate_up.restype = ctypes.c_int
    L.ep_ring_create.argtypes = [i32, i32, i32, i64]
    L.ep_ring_create.restype = P
    L.ep_ring_destroy.argtypes = [P]
    L.ep_ring_destroy.restype = ctypes.c_int
    L.ep_ring_reset.argtypes = [P]
    L.ep_ring_reset.restype = ctypes.c_int
    L.ep_ring_drain.argtypes = [P, i32, P, i32, ctypes.POINTER(i32)]
    L.ep_ring_drain.restype = ctypes.c_int
    L.ep_ring_proxy_start.argtypes = [P, i32, i64]
    L.ep_ring_proxy_start.restype = ctypes.c_int
    L.ep_ring_proxy_stop.argtypes = [P, P, i64, ctypes.POINTER(i64), ctypes.POINTER(i64)]
    L.ep_ring_proxy_stop.restype = ctypes.c_int
    L.ep_ring_proxy_drained.argtypes = [P]
    L.ep_ring_proxy_drained.restype = i64
    u64p = ctypes.POINTER(ctypes.c_uint64)
    L.ep_ring_set_loopback.argtypes = [P, P, ctypes.c_uint64, i32, ctypes.POINTER(P), u64p,
                                       ctypes.POINTER(P), u64p]
    L.ep_ring_set_loopback.restype = ctypes.c_int
    L.ep_ring_completed.argtypes = [P, i32]
    L.ep_ring_completed.restype = i64
    L.ep_ring_check_completion.argtypes = [P, P, P, i32, P, P]
    L.ep_ring_check_completion.restype = ctypes.c_int
    L.ep_ring_wait_complete.argtypes = [P, i64]
    L.ep_ring_wait_complete.restype = ctypes.c_int
    i64p = ctypes.POINTER(i64)
    dp = ctypes.POINTER(ctypes.c_double)
    L.ep_ring_loopback_stats.argtypes = [P, i64p, i64p, i64p, dp, dp]
    L.ep_ring_loopback_stats.restype = ctypes.c_int
    L.ep_status_str.argtypes = [ctypes.c_int]
    L.ep_status_str.restype = ctypes.c_char_p
    L.ep_last_error.argtypes = []
    L.ep_last_error.restype = ctypes.c_char_p
    return L


lib = _load()


def status_str(st: int) -> str:
    return lib.ep_status_str(int(st)).decode()


def _check(st: int, where: str) -> None:
    if st != EP_OK:
        raise EpError(st, where)


def shape(T: int, H: int, E: int, R: int, k: int, fmt: int = EP_FMT_BF16) -> ep_shape_t:
    return ep_shape_t(T, H, E, R, k, fmt)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def ep_row_bytes(H: int, fmt: int) -> int:
    return int(lib.ep_row_bytes(H, fmt))


def ep_workspace_bytes(s: ep_shape_t) -> int:
    return int(lib.ep_workspace_bytes(ctypes.byref(s)))


def ep_dispatch_layout(s, topk_idx, num_tokens_per_rank, num_tokens_per_expert, rank_offset,
                       expert_offset, is_token_in_rank, send_slot, workspace, dev_status,
                       stream=None) -> None:
    st = lib.ep_dispatch_layout(ctypes.byref(s), _ptr(topk_idx), _ptr(num_tokens_per_rank),
                                _ptr(num_tokens_per_expert), _ptr(rank_offset),
                                _ptr(expert_offset), _ptr(is_token_in_rank), _ptr(send_slot),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(dev_status), _stream(stream))
    _check(st, "ep_dispatch_layout")


def ep_dispatch(s, x, topk_idx, topk_w, rank_offset, send_slot, send_buf, slot_src,
                slot_local_idx, slot_local_w, ring, workspace, dev_status, stream=None,
                capacity_rows: Optional[int] = None) -> None:
    cap = send_buf.shape[0] if capacity_rows is None else capacity_rows
    st = lib.ep_dispatch(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                         _ptr(rank_offset), _ptr(send_slot), _ptr(send_buf), cap,
                         _ptr(slot_src), _ptr(slot_local_idx), _ptr(slot_local_w),
                         ring.handle if ring is not None else None, _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _ptr(dev_status),
                         _stream(stream))
    _check(st, "ep_dispatch")


def ep_dispatch_fused(s, x, topk_idx, topk_w, num_tokens_per_rank, num_tokens_per_expert,
                      rank_offset, expert_offset, is_token_in_rank, send_slot, send_buf, slot_src,
                      slot_local_idx, slot_local_w, ring, workspace, dev_status, stream=None,
                      capacity_rows: Optional[int] = None) -> None:
    cap = send_buf.shape[0] if capacity_rows is None else capacity_rows
    st = lib.ep_dispatch_fused(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                               _ptr(num_tokens_per_rank), _ptr(num_tokens_per_expert),
                               _ptr(rank_offset), _ptr(expert_offset), _ptr(is_token_in_rank),
                               _ptr(send_slot), _ptr(send_buf), cap, _ptr(slot_src),
                               _ptr(slot_local_idx), _ptr(slot_local_w),
                               ring.handle if ring is not None else None, _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(dev_status),
                               _stream(stream))
    _check(st, "ep_dispatch_fused")


def ep_dispatch_fused_plan(s, with_ring: bool = True) -> int:
    """EP_FUSED_ONE_KERNEL_SMALL, EP_FUSED_ONE_KERNEL_LARGE or
    EP_FUSED_TWO_CALLS: the path ep_dispatch_fused takes for shape s."""
    st = lib.ep_dispatch_fused_plan(ctypes.byref(s), 1 if with_ring else 0)
    if st not in (EP_FUSED_ONE_KERNEL_SMALL, EP_FUSED_ONE_KERNEL_LARGE, EP_FUSED_TWO_CALLS):
        _check(st, "ep_dispatch_fused_plan")
    return st


def ep_dispatch_fused_noalloc(s, x, topk_idx, topk_w, num_tokens_per_rank,
                              num_tokens_per_expert, rank_offset, expert_offset, is_token_in_rank,
                              send_slot, send_buf, slot_src, slot_local_idx, slot_local_w, ring,
                              dev_status, stream=None, capacity_rows: Optional[int] = None,
                              clear_scratch: bool = False) -> None:
    cap = send_buf.shape[0] if capacity_rows is None else capacity_rows
    st = lib.ep_dispatch_fused_noalloc(
        ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(num_tokens_per_rank),
        _ptr(num_tokens_per_expert), _ptr(rank_offset), _ptr(expert_offset),
        _ptr(is_token_in_rank), _ptr(send_slot), _ptr(send_buf), cap, _ptr(slot_src),
        _ptr(slot_local_idx), _ptr(slot_local_w), ring.handle if ring is not None else None,
        1 if clear_scratch else 0, _ptr(dev_status), _stream(stream))
    _check(st, "ep_dispatch_fused_noalloc")


def ep_combine(s, y, topk_idx, topk_w, send_slot, out, dev_status, stream=None) -> None:
    st = lib.ep_combine(ctypes.byref(s), _ptr(y), y.shape[0], _ptr(topk_idx), _ptr(topk_w),
                        _ptr(send_slot), _ptr(out), _ptr(dev_status), _stream(stream))
    _check(st, "ep_combine")


def ep_dispatch_layout_ll(s, topk_idx, expert_offset, expert_slot, workspace, dev_status,
                          stream=None) -> None:
    st = lib.ep_dispatch_layout_ll(ctypes.byref(s), _ptr(topk_idx), _ptr(expert_offset),
                                   _ptr(expert_slot), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ep_dispatch_layout_ll")


def ep_dispatch_ll_layout(s, topk_idx, num_tokens_per_expert, expert_offset, expert_slot,
                          workspace, dev_status, stream=None) -> None:
    st = lib.ep_dispatch_ll_layout(ctypes.byref(s), _ptr(topk_idx), _ptr(num_tokens_per_expert),
                                   _ptr(expert_offset), _ptr(expert_slot), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _ptr(dev_status), _stream(stream))
    _check(st, "ep_dispatch_ll_layout")


def ep_dispatch_ll(s, x, topk_idx, topk_w, expert_offset, expert_slot, send_buf, slot_src,
                   slot_w, ring, workspace, dev_status, stream=None,
                   capacity_rows: Optional[int] = None) -> None:
    cap = send_buf.shape[0] if capacity_rows is None else capacity_rows
    st = lib.ep_dispatch_ll(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                            _ptr(expert_offset), _ptr(expert_slot), _ptr(send_buf), cap,
                            _ptr(slot_src), _ptr(slot_w),
                            ring.handle if ring is not None else None, _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _ptr(dev_status),
                            _stream(stream))
    _check(st, "ep_dispatch_ll")


def ep_dispatch_ll_fused(s, x, topk_idx, topk_w, num_tokens_per_expert, expert_offset,
                         expert_slot, send_buf, slot_src, slot_w, ring, workspace, dev_status,
                         stream=None, capacity_rows: Optional[int] = None) -> None:
    cap = send_buf.shape[0] if capacity_rows is None else capacity_rows
    st = lib.ep_dispatch_ll_fused(ctypes.byref(s), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                                  _ptr(num_tokens_per_expert), _ptr(expert_offset),
                                  _ptr(expert_slot), _ptr(send_buf), cap, _ptr(slot_src),
                                  _ptr(slot_w), ring.handle if ring is not None else None,
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _ptr(dev_status), _stream(stream))
    _check(st, "ep_dispatch_ll_fused")


def ep_combine_ll(s, y, topk_idx, topk_w, expert_slot, out, dev_status, stream=None) -> None:
    st = lib.ep_combine_ll(ctypes.byref(s), _ptr(y), y.shape[0], _ptr(topk_idx), _ptr(topk_w),
                           _ptr(expert_slot), _ptr(out), _ptr(dev_status), _stream(stream))
    _check(st, "ep_combine_ll")


# The calls below take their sizes from the tensors, so they also check each
# tensor: type, shape, contiguity and the current device.

_U8 = _I32 = _F32 = _BF16 = _E4M3 = None   # torch types, set at the first call
_device_now = _stream_of = None            # current device; its current stream's handle


def _types() -> None:
    import torch
    global _U8, _I32, _F32, _BF16, _E4M3, _device_now, _stream_of
    _device_now, _stream_of = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream
    _U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16
    _E4M3 = torch.float8_e4m3fn


def _arg(name, t, dtype, shape_, device):
    """Address of tensor t after its checks; None for None."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape_ and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape_:
        raise ValueError(f"{name} must have shape {tuple(shape_)}, has {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current device ({device}), is on {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _need(name, t):
    if t is None:
        raise ValueError(f"{name} must not be None")
    return t


def _call_device(stream):
    """Current device and the handle of the stream (default: its current one)."""
    if _U8 is None:
        _types()
    device = _device_now()
    if stream is None:
        return device, _stream_of(device)
    if stream.device_index != device:
        raise ValueError(f"stream must be on the current device ({device}), is on "
                         f"{stream.device_index}")
    return device, stream.cuda_stream


def _row8(H: int) -> int:
    """ep_row_bytes of an 8-bit row"""
    return -(-(H + H // 32) // 128) * 128


def _workspace(t, device, needed):
    if t is None:
        raise ValueError(f"workspace of {needed} bytes needed")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on the current device ({device})")
    return t.data_ptr(), t.numel() * t.element_size()


def ep_rmsnorm(x, residual, weight, eps, residual_out=None, y=None, rows=None, rstd=None,
               stream=None) -> None:
    device, st_ = _call_device(stream)
    if _need("x", x).dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = sh = x.shape
    if H < 8 or H % 8 or (rows is not None and H % 128):
        raise EpError(EP_ERR_INVALID_ARG, "ep_rmsnorm")
    st = lib.ep_rmsnorm(
        T, H, _arg("x", x, _BF16, sh, device), _arg("residual", residual, _BF16, sh, device),
        _arg("weight", _need("weight", weight), _F32, (H,), device), eps,
        _arg("residual_out", residual_out, _BF16, sh, device), _arg("y", y, _BF16, sh, device),
        None if rows is None else _arg("rows", rows, _U8,
                                       (T, _row8(H)), device),
        _arg("rstd", rstd, _F32, (T,), device), st_)
    _check(st, "ep_rmsnorm")


def ep_rmsnorm_workspace_bytes(T: int, H: int) -> int:
    return int(lib.ep_rmsnorm_workspace_bytes(T, H))


def ep_rmsnorm_backward(r, weight, rstd, grad_y, grad_residual, grad_x, grad_weight, workspace,
                        stream=None) -> None:
    device, st_ = _call_device(stream)
    if _need("r", r).dim() != 2:
        raise ValueError("r must be [T, H]")
    T, H = sh = r.shape
    ws, ws_bytes = (None, 0) if T == 0 else _workspace(workspace, device,
                                                       ep_rmsnorm_workspace_bytes(T, H))
    st = lib.ep_rmsnorm_backward(
        T, H, _arg("r", r, _BF16, sh, device),
        _arg("weight", _need("weight", weight), _F32, (H,), device),
        _arg("rstd", _need("rstd", rstd), _F32, (T,), device),
        _arg("grad_y", _need("grad_y", grad_y), _BF16, sh, device),
        _arg("grad_residual", grad_residual, _BF16, sh, device),
        _arg("grad_x", _need("grad_x", grad_x), _BF16, sh, device),
        _arg("grad_weight", _need("grad_weight", grad_weight), _F32, (H,), device), ws, ws_bytes,
        st_)
    _check(st, "ep_rmsnorm_backward")


def ep_route_workspace_bytes(T: int, E: int) -> int:
    return int(lib.ep_route_workspace_bytes(T, E))


def _logits_type(logits) -> int:
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if logits.dtype is _F32:
        return EP_F32
    if logits.dtype is _BF16:
        return EP_BF16
    raise ValueError(f"logits must be float32 or bfloat16, are {logits.dtype}")


def ep_route(logits, token_mask, mode, topk_idx, topk_w, num_tokens_per_expert=None,
             num_tokens=None, lse=None, balance_loss=None, workspace=None, stream=None) -> None:
    device, st_ = _call_device(stream)
    kind = _logits_type(_need("logits", logits))
    if _need("topk_idx", topk_idx).dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    T, E = logits.shape
    k = topk_idx.shape[1]
    ws, ws_bytes = None, 0
    if balance_loss is not None or num_tokens is not None or num_tokens_per_expert is not None:
        ws, ws_bytes = _workspace(workspace, device, ep_route_workspace_bytes(T, E))
    st = lib.ep_route(
        T, E, k, kind, mode, _arg("logits", logits, logits.dtype, (T, E), device),
        _arg("token_mask", token_mask, _U8, (T,), device),
        _arg("topk_idx", topk_idx, _I32, (T, k), device),
        _arg("topk_w", _need("topk_w", topk_w), _F32, (T, k), device),
        _arg("num_tokens_per_expert", num_tokens_per_expert, _I32, (E,), device),
        _arg("num_tokens", num_tokens, _I32, (1,), device), _arg("lse", lse, _F32, (T,), device),
        _arg("balance_loss", balance_loss, _F32, (1,), device), ws, ws_bytes, st_)
    _check(st, "ep_route")


def ep_route_backward(logits, token_mask, mode, topk_idx, topk_w, num_tokens_per_expert,
                      num_tokens, lse, grad_topk_w, grad_balance_loss, grad_logits,
                      stream=None) -> None:
    device, st_ = _call_device(stream)
    kind = _logits_type(_need("logits", logits))
    if _need("topk_idx", topk_idx).dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    T, E = sh = logits.shape
    k = topk_idx.shape[1]
    st = lib.ep_route_backward(
        T, E, k, kind, mode, _arg("logits", logits, logits.dtype, sh, device),
        _arg("token_mask", token_mask, _U8, (T,), device),
        _arg("topk_idx", topk_idx, _I32, (T, k), device),
        _arg("topk_w", topk_w, _F32, (T, k), device),
        _arg("num_tokens_per_expert", num_tokens_per_expert, _I32, (E,), device),
        _arg("num_tokens", num_tokens, _I32, (1,), device),
        _arg("lse", _need("lse", lse), _F32, (T,), device),
        _arg("grad_topk_w", grad_topk_w, _F32, (T, k), device),
        _arg("grad_balance_loss", grad_balance_loss, _F32, (1,), device),
        _arg("grad_logits", _need("grad_logits", grad_logits), logits.dtype, sh, device), st_)
    _check(st, "ep_route_backward")


def _expert_args(rows, group_offset, w, w_scale, device):
    """G, M, weight rows, K and the addresses of the four inputs."""
    if _need("w", w).dim() != 3 or _need("rows", rows).dim() != 2:
        raise ValueError("w must be [G, N, K] and rows [M, row bytes]")
    G, N, K = w.shape
    M = rows.shape[0]
    if G < 1 or N < 1 or K < 128 or K % 128:
        raise EpError(EP_ERR_INVALID_ARG, "expert product")
    if w.dtype is not _U8 and w.dtype is not _E4M3:
        raise ValueError(f"w must be uint8 or float8_e4m3fn, is {w.dtype}")
    return (G, M, N, K,
            _arg("rows", rows, _U8, (M, _row8(K)), device),
            _arg("group_offset", _need("group_offset", group_offset), _I32, (G + 1,), device),
            _arg("w", w, w.dtype, (G, N, K), device),
            _arg("w_scale", _need("w_scale", w_scale), _F32, (G, -(-N // 128), K // 128), device))


def ep_expert_product(rows, group_offset, w, w_scale, out, dev_status, stream=None) -> None:
    device, st_ = _call_device(stream)
    G, M, N, K, *inputs = _expert_args(rows, group_offset, w, w_scale, device)
    st = lib.ep_expert_product(G, M, N, K, *inputs,
                               _arg("out", _need("out", out), _BF16, (M, N), device),
                               _arg("dev_status", _need("dev_status", dev_status), _I32, (1,),
                                    device), st_)
    _check(st, "ep_expert_product")


def ep_expert_gate_up(rows, group_offset, w, w_scale, out_rows, dev_status, stream=None) -> None:
    device, st_ = _call_device(stream)
    G, M, N, K, *inputs = _expert_args(rows, group_offset, w, w_scale, device)
    if N % 256:
        raise EpError(EP_ERR_INVALID_ARG, "ep_expert_gate_up")
    F = N // 2
    st = lib.ep_expert_gate_up(G, M, F, K, *inputs,
                               _arg("out_rows", _need("out_rows", out_rows), _U8,
                                    (M, _row8(F)), device),
                               _arg("dev_status", _need("dev_status", dev_status), _I32, (1,),
                                    device), st_)
    _check(st, "ep_expert_gate_up")


class Ring:
    """ep_ring_t: TransferCmd FIFO with `channels` channels of `depth` slots."""

    def __init__(self, depth: int = 1024, channels: int = 1, max_inflight: int = 256,
                 timeout_ns: int = 2_000_000_000):
        h = lib.ep_ring_create(depth, channels, max_inflight, timeout_ns)
        if not h:
            raise EpError(EP_ERR_INVALID_ARG, "ep_ring_create")
        self.handle = h
        self.depth, self.channels, self.max_inflight = depth, channels, max_inflight

    def destroy(self) -> None:
        if self.handle:
            _check(lib.ep_ring_destroy(self.handle), "ep_ring_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    def reset(self) -> None:
        _check(lib.ep_ring_reset(self.handle), "ep_ring_reset")

    def drain(self, channel: int, max_n: int = 1 << 16) -> np.ndarray:
        out = np.zeros(max_n, CMD_DTYPE)
        n = ctypes.c_int32(0)
        _check(lib.ep_ring_drain(self.handle, channel, out.ctypes.data, max_n, ctypes.byref(n)),
               "ep_ring_drain")
        return out[:n.value]

    def proxy_start(self, threads: int = 4, log_capacity: int = 0) -> None:
        _check(lib.ep_ring_proxy_start(self.handle, threads, log_capacity), "ep_ring_proxy_start")

    def proxy_stop(self, log_max: int = 0):
        out = np.zeros(max(log_max, 0), CMD_DTYPE)
        nl, nd = ctypes.c_int64(0), ctypes.c_int64(0)
        _check(lib.ep_ring_proxy_stop(self.handle, out.ctypes.data if log_max > 0 else None,
                                      log_max, ctypes.byref(nl), ctypes.byref(nd)),
               "ep_ring_proxy_stop")
        return out[:min(nl.value, max(log_max, 0))], nd.value

    def set_loopback(self, src, dst_list, count_list) -> None:
        """Execute popped commands against local memory: src is the send
        buffer, dst_list / count_list one device tensor (or None) per rank."""
        if src is None:
            _check(lib.ep_ring_set_loopback(self.handle, None, 0, 0, None, None, None, None),
                   "ep_ring_set_loopback")
            self._lb_keep = None
            return
        R = len(dst_list)
        P = ctypes.c_void_p
        dst = (P * R)(*[_ptr(t) for t in dst_list])
        dsz = (ctypes.c_uint64 * R)(*[0 if t is None else t.numel() * t.element_size()
                                      for t in dst_list])
        cnt = (P * R)(*[_ptr(t) for t in count_list])
        csz = (ctypes.c_uint64 * R)(*[0 if t is None else t.numel() * t.element_size()
                                      for t in count_list])
        self._lb_keep = (src, list(dst_list), list(count_list))   # keep the memory alive
        _check(lib.ep_ring_set_loopback(self.handle, _ptr(src), src.numel() * src.element_size(),
                                        R, dst, dsz, cnt, csz), "ep_ring_set_loopback")

    def completed(self, channel: int) -> int:
        return int(lib.ep_ring_completed(self.handle, channel))

    def check_completion(self, channels, tickets, done, stream=None) -> None:
        """ep_ring_check_completion: device tensors channels (int32), tickets
        (uint64 as int64) and done (uint8), all of length n."""
        _check(lib.ep_ring_check_completion(self.handle, _ptr(channels), _ptr(tickets),
                                            int(done.numel()), _ptr(done), _stream(stream)),
               "ep_ring_check_completion")

    def wait_complete(self, timeout_ns: int = 10_000_000_000) -> None:
        _check(lib.ep_ring_wait_complete(self.handle, timeout_ns), "ep_ring_wait_complete")

    def loopback_stats(self) -> dict:
        n, e, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        mean, mx = ctypes.c_double(), ctypes.c_double()
        _check(lib.ep_ring_loopback_stats(self.handle, ctypes.byref(n), ctypes.byref(e),
                                          ctypes.byref(c), ctypes.byref(mean), ctypes.byref(mx)),
               "ep_ring_loopback_stats")
        return {"completed": n.value, "errors": e.value, "copies": c.value,
                "mean_latency_us": mean.value, "max_latency_us": mx.value}

    def proxy_drained(self) -> int:
        return int(lib.ep_ring_proxy_drained(self.handle))


class Buffers:
    """Device buffers of one dispatch/combine pass for shape ``s`` (plumbing:
    torch allocations sized from the shape; nothing here computes)."""

    def __init__(self, s: ep_shape_t, capacity_rows: Optional[int] = None, device="cuda"):
        import torch
        T, H, E, R, k = s.T, s.H, s.E, s.R, s.k
        cap = T * min(k, R) if capacity_rows is None else capacity_rows
        rb = ep_row_bytes(H, s.fmt)
        i32 = dict(dtype=torch.int32, device=device)
        self.shape = s
        self.capacity_rows = cap
        self.row_bytes = rb
        self.num_tokens_per_rank = torch.empty(R, **i32)
        self.num_tokens_per_expert = torch.empty(E, **i32)
        self.rank_offset = torch.empty(R + 1, **i32)
        self.expert_offset = torch.empty(E + 1, **i32)
        self.is_token_in_rank = torch.empty((T, R), dtype=torch.uint8, device=device)
        self.send_slot = torch.empty((T, R), **i32)
        self.send_buf = torch.empty((cap, rb), dtype=torch.uint8, device=device)
        self.slot_src = torch.empty(cap, **i32)
        self.slot_local_idx = torch.empty((cap, k), **i32)
        self.slot_local_w = torch.empty((cap, k), dtype=torch.float32, device=device)
        # zero-filled once; the library keeps it consistent afterwards
        self.workspace = torch.zeros(max(ep_workspace_bytes(s), 256), dtype=torch.uint8,
                                     device=device)
        self.dev_status = torch.zeros(1, **i32)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=device)

    def layout(self, topk_idx, stream=None):
        ep_dispatch_layout(self.shape, topk_idx, self.num_tokens_per_rank,
                           self.num_tokens_per_expert, self.rank_offset, self.expert_offset,
                           self.is_token_in_rank, self.send_slot, self.workspace,
                           self.dev_status, stream)

    def dispatch(self, x, topk_idx, topk_w, ring=None, stream=None):
        ep_dispatch(self.shape, x, topk_idx, topk_w, self.rank_offset, self.send_slot,
                    self.send_buf, self.slot_src, self.slot_local_idx, self.slot_local_w, ring,
                    self.workspace, self.dev_status, stream)

    def dispatch_fused(self, x, topk_idx, topk_w, ring=None, stream=None):
        """layout + dispatch in one call (one kernel for T <= 256)"""
        ep_dispatch_fused(self.shape, x, topk_idx, topk_w, self.num_tokens_per_rank,
                          self.num_tokens_per_expert, self.rank_offset, self.expert_offset,
                          self.is_token_in_rank, self.send_slot, self.send_buf, self.slot_src,
                          self.slot_local_idx, self.slot_local_w, ring, self.workspace,
                          self.dev_status, stream)

    def dispatch_fused_noalloc(self, x, topk_idx, topk_w, ring=None, stream=None,
                               clear_scratch=False):
        """layout + dispatch in one call on the library's own device scratch
        (no workspace; the buffers' own workspace is not used)"""
        ep_dispatch_fused_noalloc(self.shape, x, topk_idx, topk_w, self.num_tokens_per_rank,
                                  self.num_tokens_per_expert, self.rank_offset,
                                  self.expert_offset, self.is_token_in_rank, self.send_slot,
                                  self.send_buf, self.slot_src, self.slot_local_idx,
                                  self.slot_local_w, ring, self.dev_status, stream,
                                  clear_scratch=clear_scratch)

    def combine(self, y, topk_idx, topk_w, stream=None):
        ep_combine(self.shape, y, topk_idx, topk_w, self.send_slot, self.out, self.dev_status,
                   stream)


class BuffersLL(Buffers):
    """Buffers of one per-expert (low-latency) pass: the rank layout's
    buffers (its counts, offsets and workspace are reused) plus the per-expert
    rows, metadata and row table.  Capacity defaults to T*k rows."""

    def __init__(self, s: ep_shape_t, capacity_rows: Optional[int] = None, device="cuda"):
        import torch
        super().__init__(s, capacity_rows=0, device=device)
        T, k = s.T, s.k
        cap = T * k if capacity_rows is None else capacity_rows
        self.capacity_rows = cap
        self.expert_slot = torch.empty((T, k), dtype=torch.int32, device=device)
        self.send_buf = torch.empty((cap, self.row_bytes), dtype=torch.uint8, device=device)
        self.slot_src = torch.empty(cap, dtype=torch.int32, device=device)
        self.slot_w = torch.empty(cap, dtype=torch.float32, device=device)

    def layout(self, topk_idx, stream=None):
        super().layout(topk_idx, stream)
        ep_dispatch_layout_ll(self.shape, topk_idx, self.expert_offset, self.expert_slot,
                              self.workspace, self.dev_status, stream)

    def layout_one_call(self, topk_idx, stream=None):
        """the per-expert layout in one kernel (ep_dispatch_ll_layout; E <=
        1024); the rank-layout buffers are left untouched"""
        ep_dispatch_ll_layout(self.shape, topk_idx, self.num_tokens_per_expert,
                              self.expert_offset, self.expert_slot, self.workspace,
                              self.dev_status, stream)

    def dispatch(self, x, topk_idx, topk_w, ring=None, stream=None):
        ep_dispatch_ll(self.shape, x, topk_idx, topk_w, self.expert_offset, self.expert_slot,
                       self.send_buf, self.slot_src, self.slot_w, ring, self.workspace,
                       self.dev_status, stream)

    def dispatch_fused(self, x, topk_idx, topk_w, ring=None, stream=None):
        """per-expert layout, row table and pack in one kernel (T <= 256,
        E <= 1024); the rank-layout buffers are left untouched"""
        ep_dispatch_ll_fused(self.shape, x, topk_idx, topk_w, self.num_tokens_per_expert,
                             self.expert_offset, self.expert_slot, self.send_buf, self.slot_src,
                             self.slot_w, ring, self.workspace, self.dev_status, stream)

    def combine(self, y, topk_idx, topk_w, stream=None):
        ep_combine_ll(self.shape, y, topk_idx, topk_w, self.expert_slot, self.out,
                      self.dev_status, stream)


class BuffersMoE(BuffersLL):
    """Buffers of a whole mixture-of-experts block over per-expert rows in 8
    bits (``s.fmt`` EP_FMT_FP8_E4M3_B128): norm, router, dispatch, the experts'
    two products of inner width ``F`` and combine, in this order.

    A serving form: ``route`` makes the choices and their gates alone.  The counts,
    the balance loss and the lse that ep_route_backward takes come from ep_route
    with a workspace."""

    def __init__(self, s: ep_shape_t, F: int, capacity_rows: Optional[int] = None, device="cuda"):
        import torch
        if s.fmt != EP_FMT_FP8_E4M3_B128:
            raise ValueError("the experts take 8-bit rows: fmt must be EP_FMT_FP8_E4M3_B128")
        super().__init__(s, capacity_rows, device)
        T, H, k, cap = s.T, s.H, s.k, self.capacity_rows
        bf, f32 = dict(dtype=torch.bfloat16, device=device), dict(dtype=torch.float32, device=device)
        self.residual = torch.empty((T, H), **bf)
        self.normed = torch.empty((T, H), **bf)
        self.rstd = torch.empty(T, **f32)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), **f32)
        self.inner = torch.empty((cap, ep_row_bytes(F, EP_FMT_FP8_E4M3_B128)), dtype=torch.uint8,
                                 device=device)
        self.y = torch.empty((cap, H), **bf)

    def norm(self, x, residual, weight, eps, stream=None):
        """self.residual = x + residual (x where residual is None, a first
        layer's) and self.normed, its norm"""
        ep_rmsnorm(x, residual, weight, eps, None if residual is None else self.residual,
                   self.normed, None, self.rstd, stream)
        if residual is None:    # the call has no residual sum to store then
            import torch
            with torch.cuda.stream(stream):
                self.residual.copy_(x)

    def route(self, logits, mode=EP_GATE_SOFTMAX_RENORM, token_mask=None, stream=None):
        ep_route(logits, token_mask, mode, self.topk_idx, self.topk_w, stream=stream)

    def experts(self, w_gate_up, gate_up_scale, w_down, down_scale, stream=None):
        """self.y = the experts' outputs for the rows in self.send_buf"""
        ep_expert_gate_up(self.send_buf, self.expert_offset, w_gate_up, gate_up_scale, self.inner,
                          self.dev_status, stream)
        ep_expert_product(self.inner, self.expert_offset, w_down, down_scale, self.y,
                          self.dev_status, stream)

    def block(self, x, residual, weight, eps, router, w_gate_up, gate_up_scale, w_down, down_scale,
              mode=EP_GATE_SOFTMAX_RENORM, token_mask=None):
        """The whole block on the current stream; router(normed) gives the
        logits [T, E].  Returns the combined output; self.residual is the
        residual stream that it belongs to."""
        self.norm(x, residual, weight, eps)
        self.route(router(self.normed), mode, token_mask)
        self.layout(self.topk_idx)
        self.dispatch(self.normed, self.topk_idx, self.topk_w)
        self.experts(w_gate_up, gate_up_scale, w_down, down_scale)
        self.combine(self.y, self.topk_idx, self.topk_w)
        return self.out
