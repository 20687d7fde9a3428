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
    ep_combine_backward(shape, y, topk_idx, topk_w, send_slot, grad_out, grad_y, grad_topk_w,
                        dev_status, stream=None)             # ep_combine_ll_backward: expert_slot
    ep_dispatch_backward(shape, topk_idx, send_slot, grad_rows, grad_slot_local_w, grad_other,
                         grad_x, grad_topk_w, dev_status, stream=None)
        (ep_dispatch_ll_backward: expert_slot and grad_slot_w)
    ep_expert_product_bf16(rows, group_offset, w, out, dev_status, stream=None)
    ep_expert_product_bf16_backward(rows, group_offset, w, grad_out, grad_rows, grad_w, dev_status,
                                    workspace=None, stream=None)
    ep_expert_gate_up_bf16(rows, group_offset, w, pre, out, dev_status, stream=None)
    ep_expert_gate_up_bf16_backward(rows, group_offset, w, pre, grad_out, grad_pre, grad_rows,
                                    grad_w, dev_status, workspace=None, stream=None)
    ep_expert_bf16_plan(product, G, M, N, K)   # the tiles that one of the EP_PRODUCT_* takes
    ep_grad_norm(tensors, sum_squares, norm, workspace, stream=None)
    ep_grad_clip(tensors, sum_squares, max_norm, into=None, stream=None)
        (these take their sizes from the tensors, or check them against the shape: a wrong
        type, shape, device or stride raises ValueError)
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
EP_PRODUCT_FORWARD = 0
EP_PRODUCT_GATE_UP = 1
EP_PRODUCT_ROWS_BACKWARD = 2
EP_PRODUCT_WEIGHTS_BACKWARD = 3
EP_TILES_SMALL = 111
EP_TILES_BIG = 112
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


class ep_tensor_t(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("pad_", ctypes.c_int32)]


class ep_tensor_list_t(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("units", ctypes.c_int64), ("sizes", ctypes.c_uint64),
                ("count", ctypes.c_int32), ("pad_", ctypes.c_int32)]


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
    L.ep_combine_backward.argtypes = [S, P, i64, P, P, P, P, P, P, P, P]
    L.ep_combine_backward.restype = ctypes.c_int
    L.ep_combine_ll_backward.argtypes = L.ep_combine_backward.argtypes
    L.ep_combine_ll_backward.restype = ctypes.c_int
    L.ep_dispatch_backward.argtypes = [S, P, P, P, i64, P, P, P, P, P, P]
    L.ep_dispatch_backward.restype = ctypes.c_int
    L.ep_dispatch_ll_backward.argtypes = L.ep_dispatch_backward.argtypes
    L.ep_dispatch_ll_backward.restype = ctypes.c_int
    L.ep_expert_product_bf16.argtypes = [i32, i64, i32, i32, P, P, P, P, P, P]
    L.ep_expert_product_bf16.restype = ctypes.c_int
    L.ep_expert_gate_up_bf16.argtypes = [i32, i64, i32, i32, P, P, P, P, P, P, P]
    L.ep_expert_gate_up_bf16.restype = ctypes.c_int
    L.ep_expert_bf16_plan.argtypes = [i32, i32, i64, i32, i32]
    L.ep_expert_bf16_plan.restype = ctypes.c_int
    L.ep_expert_backward_workspace_bytes.argtypes = [i32, i64, i32, i32]
    L.ep_expert_backward_workspace_bytes.restype = sz
    L.ep_expert_product_bf16_backward.argtypes = [i32, i64, i32, i32, i32, P, P, P, P, P, P, P, P,
                                                  sz, P]
    L.ep_expert_product_bf16_backward.restype = ctypes.c_int
    L.ep_expert_gate_up_bf16_backward.argtypes = [i32, i64, i32, i32, i32, P, P, P, P, P, P, P, P,
                                                  P, P, sz, P]
    L.ep_expert_gate_up_bf16_backward.restype = ctypes.c_int
    TL = ctypes.POINTER(ep_tensor_list_t)
    L.ep_tensor_table_bytes.argtypes = [i32]
    L.ep_tensor_table_bytes.restype = sz
    L.ep_tensor_table.argtypes = [i32, ctypes.POINTER(ep_tensor_t), P, TL]
    L.ep_tensor_table.restype = ctypes.c_int
    L.ep_grad_norm_workspace_bytes.argtypes = []
    L.ep_grad_norm_workspace_bytes.restype = sz
    L.ep_grad_norm.argtypes = [TL, P, P, P, sz, P]
    L.ep_grad_norm.restype = ctypes.c_int
    L.ep_grad_clip.argtypes = [TL, TL, P, ctypes.c_double, P]
    L.ep_grad_clip.restype = ctypes.c_int
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

_U8 = _I32 = _F32 = _F64 = _BF16 = _E4M3 = None   # torch types, set at the first call
_device_now = _stream_of = None            # current device; its current stream's handle


def _types() -> None:
    import torch
    global _U8, _I32, _F32, _F64, _BF16, _E4M3, _device_now, _stream_of
    _device_now, _stream_of = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream
    _U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16
    _E4M3, _F64 = torch.float8_e4m3fn, torch.float64


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


def _slots(s, name, slot, topk_idx, device, ll):
    """Addresses of topk_idx and of the layout's slots, [T, R] or, per expert, [T, k]."""
    return (_arg("topk_idx", _need("topk_idx", topk_idx), _I32, (s.T, s.k), device),
            _arg(name, _need(name, slot), _I32, (s.T, s.k if ll else s.R), device))


def _status(dev_status, device):
    return _arg("dev_status", _need("dev_status", dev_status), _I32, (1,), device)


def _rows_of(s, name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, H]")
    return t.shape[0]


def _combine_backward(call, where, ll, s, y, topk_idx, topk_w, slot_name, slot, grad_out, grad_y,
                      grad_topk_w, dev_status, stream) -> None:
    device, st_ = _call_device(stream)
    if grad_y is None and grad_topk_w is None:
        raise ValueError("one of grad_y and grad_topk_w must be given")
    if grad_topk_w is not None:
        _need("y", y)
    rows = _rows_of(s, "y", y) if y is not None else _rows_of(s, "grad_y", grad_y)
    idx, slots = _slots(s, slot_name, slot, topk_idx, device, ll)
    st = call(ctypes.byref(s), _arg("y", y, _BF16, (rows, s.H), device), rows, idx,
              _arg("topk_w", _need("topk_w", topk_w), _F32, (s.T, s.k), device), slots,
              _arg("grad_out", _need("grad_out", grad_out), _BF16, (s.T, s.H), device),
              _arg("grad_y", grad_y, _BF16, (rows, s.H), device),
              _arg("grad_topk_w", grad_topk_w, _F32, (s.T, s.k), device),
              _status(dev_status, device), st_)
    _check(st, where)


def ep_combine_backward(s, y, topk_idx, topk_w, send_slot, grad_out, grad_y, grad_topk_w,
                        dev_status, stream=None) -> None:
    _combine_backward(lib.ep_combine_backward, "ep_combine_backward", False, s, y, topk_idx, topk_w,
                      "send_slot", send_slot, grad_out, grad_y, grad_topk_w, dev_status, stream)


def ep_combine_ll_backward(s, y, topk_idx, topk_w, expert_slot, grad_out, grad_y, grad_topk_w,
                           dev_status, stream=None) -> None:
    _combine_backward(lib.ep_combine_ll_backward, "ep_combine_ll_backward", True, s, y, topk_idx,
                      topk_w, "expert_slot", expert_slot, grad_out, grad_y, grad_topk_w, dev_status,
                      stream)


def _dispatch_backward(call, where, ll, s, topk_idx, slot_name, slot, grad_rows, gates_name, gates,
                       grad_other, grad_x, grad_topk_w, dev_status, stream) -> None:
    device, st_ = _call_device(stream)
    rows = _rows_of(s, "grad_rows", _need("grad_rows", grad_rows))
    if (gates is None) != (grad_topk_w is None):
        raise ValueError(f"{gates_name} and grad_topk_w belong together")
    idx, slots = _slots(s, slot_name, slot, topk_idx, device, ll)
    st = call(ctypes.byref(s), idx, slots, _arg("grad_rows", grad_rows, _BF16, (rows, s.H), device),
              rows, _arg(gates_name, gates, _F32, (rows,) if ll else (rows, s.k), device),
              _arg("grad_other", grad_other, _BF16, (s.T, s.H), device),
              _arg("grad_x", _need("grad_x", grad_x), _BF16, (s.T, s.H), device),
              _arg("grad_topk_w", grad_topk_w, _F32, (s.T, s.k), device),
              _status(dev_status, device), st_)
    _check(st, where)


def ep_dispatch_backward(s, topk_idx, send_slot, grad_rows, grad_slot_local_w, grad_other, grad_x,
                         grad_topk_w, dev_status, stream=None) -> None:
    _dispatch_backward(lib.ep_dispatch_backward, "ep_dispatch_backward", False, s, topk_idx,
                       "send_slot", send_slot, grad_rows, "grad_slot_local_w", grad_slot_local_w,
                       grad_other, grad_x, grad_topk_w, dev_status, stream)


def ep_dispatch_ll_backward(s, topk_idx, expert_slot, grad_rows, grad_slot_w, grad_other, grad_x,
                            grad_topk_w, dev_status, stream=None) -> None:
    _dispatch_backward(lib.ep_dispatch_ll_backward, "ep_dispatch_ll_backward", True, s, topk_idx,
                       "expert_slot", expert_slot, grad_rows, "grad_slot_w", grad_slot_w,
                       grad_other, grad_x, grad_topk_w, dev_status, stream)


def _bf16_args(rows, group_offset, w, device, weights=None, width=None):
    """G, M, weight rows, K and the addresses of rows, offsets and w.  In a backward
    rows or w may be None: the sizes then come from grad_w (`weights`) or grad_out."""
    sized = w if w is not None else _need("w", weights)
    if sized.dim() != 3:
        raise ValueError("w must be [G, N, K]")
    G, N, K = sized.shape
    counted = rows if rows is not None else _need("rows", width)
    if counted.dim() != 2:
        raise ValueError("rows and grad_out must be [M, K] and [M, N]")
    M = counted.shape[0]
    return (G, M, N, K, _arg("rows", rows, _BF16, (M, K), device),
            _arg("group_offset", _need("group_offset", group_offset), _I32, (G + 1,), device),
            _arg("w", w, _BF16, (G, N, K), device))


def ep_expert_product_bf16(rows, group_offset, w, out, dev_status, stream=None) -> None:
    device, st_ = _call_device(stream)
    G, M, N, K, *inputs = _bf16_args(_need("rows", rows), group_offset, _need("w", w), device)
    st = lib.ep_expert_product_bf16(G, M, N, K, *inputs,
                                    _arg("out", _need("out", out), _BF16, (M, N), device),
                                    _status(dev_status, device), st_)
    _check(st, "ep_expert_product_bf16")


def ep_expert_gate_up_bf16(rows, group_offset, w, pre, out, dev_status, stream=None) -> None:
    device, st_ = _call_device(stream)
    G, M, N, K, *inputs = _bf16_args(_need("rows", rows), group_offset, _need("w", w), device)
    if N % 16:
        raise EpError(EP_ERR_INVALID_ARG, "ep_expert_gate_up_bf16")
    st = lib.ep_expert_gate_up_bf16(G, M, N // 2, K, *inputs,
                                    _arg("pre", pre, _BF16, (M, N), device),
                                    _arg("out", _need("out", out), _BF16, (M, N // 2), device),
                                    _status(dev_status, device), st_)
    _check(st, "ep_expert_gate_up_bf16")


def ep_expert_bf16_plan(product: int, G: int, M: int, N: int, K: int) -> int:
    """EP_TILES_SMALL or EP_TILES_BIG: the tiles that one of the EP_PRODUCT_* products of rows
    [M, K] and weights [G, N, K] takes."""
    st = lib.ep_expert_bf16_plan(product, G, M, N, K)
    if st not in (EP_TILES_SMALL, EP_TILES_BIG):
        _check(st, "ep_expert_bf16_plan")
    return st


def ep_expert_backward_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    return int(lib.ep_expert_backward_workspace_bytes(G, M, N, K))


def _weights_type(grad_w) -> int:
    if grad_w is None or grad_w.dtype is _BF16:
        return EP_BF16
    if grad_w.dtype is _F32:
        return EP_F32
    raise ValueError(f"grad_w must be float32 or bfloat16, is {grad_w.dtype}")


def _backward_outputs(G, M, N, K, grad_rows, grad_w, dev_status, workspace, device):
    """The addresses of grad_rows, grad_w, dev_status and the workspace, and its bytes."""
    ws, ws_bytes = None, 0
    if grad_w is not None:
        needed = ep_expert_backward_workspace_bytes(G, M, N, K)
        if needed:
            ws, ws_bytes = _workspace(workspace, device, needed)
    return (_arg("grad_rows", grad_rows, _BF16, (M, K), device),
            None if grad_w is None else _arg("grad_w", grad_w, grad_w.dtype, (G, N, K), device),
            _status(dev_status, device), ws, ws_bytes)


def ep_expert_product_bf16_backward(rows, group_offset, w, grad_out, grad_rows, grad_w, dev_status,
                                    workspace=None, stream=None) -> None:
    device, st_ = _call_device(stream)
    if grad_rows is None and grad_w is None:
        raise ValueError("one of grad_rows and grad_w must be given")
    if grad_rows is not None:
        _need("w", w)
    if grad_w is not None:
        _need("rows", rows)
    G, M, N, K, *inputs = _bf16_args(rows, group_offset, w, device, grad_w,
                                     _need("grad_out", grad_out))
    st = lib.ep_expert_product_bf16_backward(
        G, M, N, K, _weights_type(grad_w), *inputs,
        _arg("grad_out", grad_out, _BF16, (M, N), device),
        *_backward_outputs(G, M, N, K, grad_rows, grad_w, dev_status, workspace, device), st_)
    _check(st, "ep_expert_product_bf16_backward")


def ep_expert_gate_up_bf16_backward(rows, group_offset, w, pre, grad_out, grad_pre, grad_rows,
                                    grad_w, dev_status, workspace=None, stream=None) -> None:
    device, st_ = _call_device(stream)
    G, M, N, K, *inputs = _bf16_args(_need("rows", rows), group_offset, _need("w", w), device)
    if N % 16:
        raise EpError(EP_ERR_INVALID_ARG, "ep_expert_gate_up_bf16_backward")
    st = lib.ep_expert_gate_up_bf16_backward(
        G, M, N // 2, K, _weights_type(grad_w), *inputs,
        _arg("pre", _need("pre", pre), _BF16, (M, N), device),
        _arg("grad_out", _need("grad_out", grad_out), _BF16, (M, N // 2), device),
        _arg("grad_pre", _need("grad_pre", grad_pre), _BF16, (M, N), device),
        *_backward_outputs(G, M, N, K, grad_rows, grad_w, dev_status, workspace, device), st_)
    _check(st, "ep_expert_gate_up_bf16_backward")


class TensorList:
    """Tensors of float32 and bfloat16 on the current device, as ep_grad_norm and ep_grad_clip
    take them.  Made once for gradients that keep their memory from step to step (a table goes to
    the GPU, and is waited for); it holds that memory, so a tensor that is given other memory
    (``t.data = ...``) needs a new list.  Tensors that overlap are refused."""

    def __init__(self, tensors):
        import torch
        if _U8 is None:
            _types()
        keep = [t.detach() for t in tensors]
        self.device = _device_now()
        spans = []
        for i, t in enumerate(keep):
            if t.dtype is not _F32 and t.dtype is not _BF16:
                raise ValueError(f"tensor {i} must be float32 or bfloat16, is {t.dtype}")
            if t.get_device() != self.device:
                raise ValueError(f"tensor {i} must be on the current device ({self.device}), is "
                                 f"on {t.device}")
            if not t.is_contiguous():
                raise ValueError(f"tensor {i} must be contiguous")
            if t.numel():
                spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i))
        spans.sort()
        for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"tensors {i} and {j} overlap")
        count = len(keep)
        array = (ep_tensor_t * max(1, count))(
            *[ep_tensor_t(t.data_ptr() if t.numel() else None, t.numel(),
                          EP_F32 if t.dtype is _F32 else EP_BF16, 0) for t in keep])
        table = torch.empty(int(lib.ep_tensor_table_bytes(count)), dtype=torch.uint8)
        self.c = ep_tensor_list_t()
        _check(lib.ep_tensor_table(count, array, table.data_ptr(), ctypes.byref(self.c)),
               "ep_tensor_table")
        self.tensors = keep
        self.table = table.to(torch.device("cuda", self.device))
        self.c.table = self.table.data_ptr()

    def __len__(self) -> int:
        return len(self.tensors)


def _tensor_list(tensors, device, stream, name) -> TensorList:
    if not isinstance(tensors, TensorList):
        tensors = TensorList(tensors)
        if stream is not None:      # its table outlives the call there
            tensors.table.record_stream(stream)
    if tensors.device != device:
        raise ValueError(f"{name} must be on the current device ({device}), are on "
                         f"{tensors.device}")
    return tensors


def ep_grad_norm_workspace_bytes(tensors=None) -> int:
    """The same for any list."""
    return int(lib.ep_grad_norm_workspace_bytes())


def _sum_squares(t, device):
    return _arg("sum_squares", _need("sum_squares", t), _F64, (1,), device)


def ep_grad_norm(tensors, sum_squares, norm, workspace, stream=None) -> None:
    """tensors: a TensorList, or a sequence of tensors, for which one is made (not under graph
    capture: it waits for its table)."""
    device, st_ = _call_device(stream)
    tensors = _tensor_list(tensors, device, stream, "tensors")
    ws, ws_bytes = _workspace(workspace, device, ep_grad_norm_workspace_bytes())
    st = lib.ep_grad_norm(ctypes.byref(tensors.c), _sum_squares(sum_squares, device),
                          _arg("norm", norm, _F32, (1,), device), ws, ws_bytes, st_)
    _check(st, "ep_grad_norm")


def ep_grad_clip(tensors, sum_squares, max_norm, into=None, stream=None) -> None:
    """tensors and into as at ep_grad_norm."""
    device, st_ = _call_device(stream)
    tensors = _tensor_list(tensors, device, stream, "tensors")
    into_c = None
    if into is not None:
        into = _tensor_list(into, device, stream, "into")
        if len(into) != len(tensors):
            raise ValueError(f"into must have {len(tensors)} tensors, has {len(into)}")
        into_c = ctypes.byref(into.c)
    st = lib.ep_grad_clip(ctypes.byref(tensors.c), into_c, _sum_squares(sum_squares, device),
                          max_norm, st_)
    _check(st, "ep_grad_clip")


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
                self.residual.copy_(x.detach())    # no part of x's graph

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


class BuffersMoETrain(BuffersLL):
    """Buffers of a mixture-of-experts block's training pass over per-expert rows in bf16
    (``s.fmt`` EP_FMT_BF16): norm, router with its balance loss, dispatch, the experts' two
    products of inner width ``F`` and combine, and their gradients in the opposite order.
    ``weights_dtype``: that of the experts' weights' gradients, bfloat16 or float32.

    ``forward`` and ``backward`` run on the current stream.  A backward belongs to the forward
    before it and uses up what that left (self.y and self.pre get their gradients)."""

    def __init__(self, s: ep_shape_t, F: int, capacity_rows: Optional[int] = None,
                 weights_dtype=None, device="cuda"):
        import torch
        if s.fmt != EP_FMT_BF16:
            raise ValueError("the experts take bf16 rows: fmt must be EP_FMT_BF16")
        if weights_dtype not in (None, torch.bfloat16, torch.float32):
            raise ValueError(f"weights_dtype must be float32 or bfloat16, is {weights_dtype}")
        super().__init__(s, capacity_rows, device)
        T, H, E, k, cap = s.T, s.H, s.E, s.k, self.capacity_rows
        bf = dict(dtype=torch.bfloat16, device=device)
        f32, i32 = dict(dtype=torch.float32, device=device), dict(dtype=torch.int32, device=device)
        wt = dict(dtype=weights_dtype or torch.bfloat16, device=device)
        self.F = F
        self.residual = torch.empty((T, H), **bf)
        self.normed = torch.empty((T, H), **bf)
        self.rstd = torch.empty(T, **f32)
        self.topk_idx = torch.empty((T, k), **i32)
        self.topk_w = torch.empty((T, k), **f32)
        self.num_choices = torch.empty(E, **i32)
        self.num_tokens = torch.empty(1, **i32)
        self.lse = torch.empty(T, **f32)
        self.balance_loss = torch.empty(1, **f32)
        self.rows = self.send_buf.view(torch.bfloat16)      # [cap, H]
        self.pre = torch.empty((cap, 2 * F), **bf)
        self.inner = torch.empty((cap, F), **bf)
        self.y = torch.empty((cap, H), **bf)
        self.grad_topk_w = torch.empty((T, k), **f32)
        self.grad_inner = torch.empty((cap, F), **bf)
        self.grad_rows = torch.empty((cap, H), **bf)
        self.grad_normed = torch.empty((T, H), **bf)
        self.grad_x = torch.empty((T, H), **bf)
        self.grad_weight = torch.empty(H, **f32)
        self.grad_gate_up = torch.empty((E, 2 * F, H), **wt)
        self.grad_down = torch.empty((E, H, F), **wt)
        u8 = dict(dtype=torch.uint8, device=device)
        self.route_workspace = torch.zeros(max(16, ep_route_workspace_bytes(T, E)), **u8)
        self.back_workspace = torch.empty(
            max(16, ep_rmsnorm_workspace_bytes(T, H),
                ep_expert_backward_workspace_bytes(E, cap, 2 * F, H),
                ep_expert_backward_workspace_bytes(E, cap, H, F)), **u8)
        self._saved = None

    def forward(self, x, residual, weight, eps, router, w_gate_up, w_down,
                mode=EP_GATE_SOFTMAX_RENORM, token_mask=None):
        """router(normed) gives the logits [T, E] (bf16 or float32).  Returns the combined
        output; self.residual is the residual stream that it belongs to, self.balance_loss the
        balance loss."""
        self._saved = None      # one that ends early leaves no forward to go back from
        ep_rmsnorm(x, residual, weight, eps, None if residual is None else self.residual,
                   self.normed, None, self.rstd)
        if residual is None:
            self.residual.copy_(x.detach())    # no part of x's graph
        logits = router(self.normed)
        ep_route(logits, token_mask, mode, self.topk_idx, self.topk_w, self.num_choices,
                 self.num_tokens, self.lse, self.balance_loss, self.route_workspace)
        self.layout(self.topk_idx)
        self.dispatch(self.normed, self.topk_idx, self.topk_w)
        ep_expert_gate_up_bf16(self.rows, self.expert_offset, w_gate_up, self.pre, self.inner,
                               self.dev_status)
        ep_expert_product_bf16(self.inner, self.expert_offset, w_down, self.y, self.dev_status)
        self.combine(self.y, self.topk_idx, self.topk_w)
        self._saved = (weight, w_gate_up, w_down, mode, token_mask, logits)
        return self.out

    def backward(self, grad_out, grad_residual=None, grad_balance_loss=None, router_backward=None):
        """grad_out bf16 [T, H]; grad_residual that of self.residual, grad_balance_loss (float32
        [1], on the device) that of self.balance_loss, or None.  router_backward(grad_logits)
        gives the gradient of router's input, bf16 [T, H], or None; if it raises, or gives another
        tensor, the forward is used up.  Returns the gradient of x (and of residual); the weights'
        are self.grad_weight, self.grad_gate_up and self.grad_down."""
        import torch
        if self._saved is None:
            raise RuntimeError("backward() needs a forward() before it")
        weight, w_gate_up, w_down, mode, token_mask, logits = self._saved
        s, off = self.shape, self.expert_offset
        # Every gradient that is given, before the first launch: y and pre become their own
        # gradients, and a call that is refused later would have used the forward up.
        device, _ = _call_device(None)
        _arg("grad_residual", grad_residual, _BF16, (s.T, s.H), device)
        _arg("grad_balance_loss", grad_balance_loss, _F32, (1,), device)
        ep_combine_ll_backward(s, self.y, self.topk_idx, self.topk_w, self.expert_slot, grad_out,
                               self.y, self.grad_topk_w, self.dev_status)
        self._saved = None      # not before: a refused gradient leaves the forward as it was
        ep_expert_product_bf16_backward(self.inner, off, w_down, self.y, self.grad_inner,
                                        self.grad_down, self.dev_status, self.back_workspace)
        ep_expert_gate_up_bf16_backward(self.rows, off, w_gate_up, self.pre, self.grad_inner,
                                        self.pre, self.grad_rows, self.grad_gate_up,
                                        self.dev_status, self.back_workspace)
        grad_logits = torch.empty_like(logits)
        ep_route_backward(logits, token_mask, mode, self.topk_idx, self.topk_w, self.num_choices,
                          self.num_tokens, self.lse, self.grad_topk_w, grad_balance_loss,
                          grad_logits)
        other = router_backward(grad_logits) if router_backward is not None else None
        ep_dispatch_ll_backward(s, self.topk_idx, self.expert_slot, self.grad_rows, None, other,
                                self.grad_normed, None, self.dev_status)
        ep_rmsnorm_backward(self.residual, weight, self.rstd, self.grad_normed, grad_residual,
                            self.grad_x, self.grad_weight, self.back_workspace)
        return self.grad_x

    def gradients(self):
        """The weights' gradients, as ep_grad_norm and ep_grad_clip take them."""
        return TensorList([self.grad_weight, self.grad_gate_up, self.grad_down])
