"""Thin Python binding of the C ABI in include/moe.h (libmoe_gb300.so).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch supplies device memory and
the current stream); the functions carry the C names.  If the library has not
been built the first call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import numpy as np
import torch

from . import build as _build

MOE_F32, MOE_BF16, MOE_Q8_0, MOE_Q4_A64, MOE_Q4_K, MOE_Q6_K, MOE_FP8 = 0, 1, 2, 3, 4, 5, 6
PACKED = (MOE_Q8_0, MOE_Q4_A64, MOE_Q4_K, MOE_Q6_K, MOE_FP8)   # storage types moe_forward takes repacked
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL, MOE_PATH_DECODE_SIMT = 0, 1, 2, 3
MOE_SCORE_SELECTED_SOFTMAX, MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1, 2
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
          6: "MOE_ERR_DEVICE_CHECK"}

# Every symbol include/moe.h declares.
EXPORTS = ("moe_status_str", "moe_version", "moe_route", "moe_route_scored", "moe_permute",
           "moe_q8_0_packed_size", "moe_pack_q8_0", "moe_q4_a64_packed_size", "moe_pack_q4_a64",
           "moe_q4_k_packed_size", "moe_pack_q4_k", "moe_q6_k_packed_size", "moe_pack_q6_k",
           "moe_fp8_packed_size", "moe_pack_fp8",
           "moe_workspace_size", "moe_forward",
           "moe_forward_profiled", "moe_forward_scored", "moe_ffn_dense", "moe_forward_noalloc",
           "moe_workspace_views", "moe_forward_expire_wait", "moe_check", "moe_check_noalloc",
           "moe_quant_fp8b", "moe_norm_fp8b", "moe_gemm_fp8b", "moe_grouped_gemm_fp8b",
           "moe_gate_up_fp8b", "moe_fp8b_workspace_size", "moe_grouped_gemm_fp8b_expire_wait",
           "moe_grouped_gemm_fp8b_expire_sums", "moe_gate_up_fp8b_expire_wait",
           "moe_gate_up_fp8b_expire_sums",
           "moe_dispatch", "moe_dispatch_filled", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
           "moe_combine_backward_filled", "moe_quant_i8", "moe_gemm_i8", "moe_grouped_gemm_i8", "moe_gate_up_i8", "moe_i8_workspace_size",
           "moe_grouped_gemm_i8_expire_wait", "moe_gate_up_i8_expire_wait")

_lib = None
_debug_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({_lib.moe_status_str(status).decode() if _lib else ''})")


def library_path() -> str:
    return _build.LIB_PATH


def load_library():
    """Load libmoe_gb300.so and declare its signatures (raises if missing)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the CUDA library first "
            "(python -m expert_routed_ffn_selectedsoftmax_gb300.build)")
    _lib = _declare(ctypes.CDLL(path))
    return _lib


def load_debug_library():
    """The debug build (libmoe_gb300_debug.so, MOE_DEBUG=1: device-side checks
    of the grouping the expert kernels are given; include/moe_debug.h),
    compiled first if it is missing or stale.  A separate ctypes handle with
    the same signatures plus moe_debug_corrupt_next_offsets; the functions of
    this module keep using the release library."""
    global _debug_lib
    if _debug_lib is None:
        L = _declare(ctypes.CDLL(_build.build(debug=True)))
        L.moe_debug_corrupt_next_offsets.argtypes = []
        L.moe_debug_corrupt_next_offsets.restype = ctypes.c_int
        _debug_lib = L
    return _debug_lib


def _declare(L):
    vp, i, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
    L.moe_status_str.argtypes = [i]
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_version.argtypes = []
    L.moe_version.restype = i
    L.moe_route.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp]
    L.moe_route.restype = i
    L.moe_route_scored.argtypes = [vp, i, i, i, vp, vp, i, i, i, vp, vp, vp]
    L.moe_route_scored.restype = i
    L.moe_permute.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp]
    L.moe_permute.restype = i
    L.moe_q8_0_packed_size.argtypes = [ll, i]
    L.moe_q8_0_packed_size.restype = sz
    L.moe_pack_q8_0.argtypes = [vp, ll, i, vp, vp]
    L.moe_pack_q8_0.restype = i
    L.moe_q4_a64_packed_size.argtypes = [ll, i]
    L.moe_q4_a64_packed_size.restype = sz
    L.moe_pack_q4_a64.argtypes = [vp, ll, i, vp, vp]
    L.moe_pack_q4_a64.restype = i
    L.moe_q4_k_packed_size.argtypes = [ll, i]
    L.moe_q4_k_packed_size.restype = sz
    L.moe_pack_q4_k.argtypes = [vp, ll, i, vp, vp]
    L.moe_pack_q4_k.restype = i
    L.moe_q6_k_packed_size.argtypes = [ll, i]
    L.moe_q6_k_packed_size.restype = sz
    L.moe_pack_q6_k.argtypes = [vp, ll, i, vp, vp]
    L.moe_pack_q6_k.restype = i
    L.moe_fp8_packed_size.argtypes = [ll, i]
    L.moe_fp8_packed_size.restype = sz
    L.moe_pack_fp8.argtypes = [vp, ll, i, vp, vp]
    L.moe_pack_fp8.restype = i
    L.moe_workspace_size.argtypes = [i, i, i, i, i, i, i]
    L.moe_workspace_size.restype = sz
    L.moe_forward.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp, i, i, vp, vp, sz, i, vp]
    L.moe_forward.restype = i
    L.moe_forward_profiled.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp, i, i, vp, vp, sz,
                                       i, vp, vp]
    L.moe_forward_profiled.restype = i
    L.moe_forward_scored.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp, i, i, vp, vp, sz,
                                     i, i, vp, vp]
    L.moe_forward_scored.restype = i
    L.moe_ffn_dense.argtypes = [vp, i, i, i, vp, vp, vp, i, i, vp, vp, sz, i, vp]
    L.moe_ffn_dense.restype = i
    L.moe_forward_noalloc.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp, i, i, vp, i, vp]
    L.moe_forward_noalloc.restype = i
    L.moe_forward_expire_wait.argtypes = [vp, i, i, i, vp, vp, i, i, vp, vp, vp, i, i, vp, vp, sz,
                                          i, i, ctypes.c_uint32, vp]
    L.moe_forward_expire_wait.restype = i
    L.moe_workspace_views.argtypes = [i, i, i, i, i, i, i, vp]
    L.moe_workspace_views.restype = i
    f = ctypes.c_float
    L.moe_quant_fp8b.argtypes = [vp, i, i, i, i, ll, i, vp, vp, vp]
    L.moe_quant_fp8b.restype = i
    L.moe_norm_fp8b.argtypes = [vp, i, i, i, ll, vp, i, i, ll, vp, vp, i, vp, i, f, vp, vp, vp, vp,
                                vp]
    L.moe_norm_fp8b.restype = i
    L.moe_gemm_fp8b.argtypes = [vp, vp, i, i, ll, vp, vp, i, vp, i, ll, vp, vp]
    L.moe_gemm_fp8b.restype = i
    L.moe_grouped_gemm_fp8b.argtypes = [vp, vp, i, i, ll, vp, vp, i, i, vp, vp, i, vp, i, ll, vp,
                                        sz, vp, vp]
    for hook in (L.moe_grouped_gemm_fp8b_expire_wait, L.moe_grouped_gemm_fp8b_expire_sums):
        hook.argtypes = [vp, vp, i, i, ll, vp, vp, i, i, vp, vp, i, vp, i, ll, vp, sz, vp, ctypes.c_uint32, vp]
        hook.restype = i
    for hook in (L.moe_gate_up_fp8b_expire_wait, L.moe_gate_up_fp8b_expire_sums):
        hook.argtypes = [vp, vp, i, i, ll, vp, vp, vp, vp, i, i, vp, vp, i, vp, vp, vp, sz, vp,
                         ctypes.c_uint32, vp]
        hook.restype = i
    L.moe_fp8b_workspace_size.argtypes = [i, i]
    L.moe_fp8b_workspace_size.restype = sz
    L.moe_grouped_gemm_fp8b.restype = i
    L.moe_gate_up_fp8b.argtypes = [vp, vp, i, i, ll, vp, vp, vp, vp, i, i, vp, vp, i, vp, vp, vp,
                                   sz, vp, vp]
    L.moe_gate_up_fp8b.restype = i
    L.moe_dispatch.argtypes = [vp, i, i, i, ll, vp, i, vp, i, ll, vp]
    L.moe_dispatch_filled.argtypes = L.moe_dispatch.argtypes
    L.moe_dispatch_backward.argtypes = [vp, i, i, i, ll, vp, i, i, vp, ll, vp]
    L.moe_combine.argtypes = [vp, i, i, i, ll, vp, vp, i, i, vp, i, ll, vp]
    L.moe_combine_backward.argtypes = [vp, i, i, i, ll, vp, i, i, ll, vp, vp, i, vp, ll, vp, vp]
    L.moe_combine_backward_filled.argtypes = L.moe_combine_backward.argtypes
    L.moe_quant_i8.argtypes = [vp, i, i, i, ll, vp, vp, vp]
    L.moe_gemm_i8.argtypes = [vp, vp, i, i, ll, vp, vp, i, vp, i, ll, vp, sz, vp, vp]
    L.moe_grouped_gemm_i8.argtypes = [vp, vp, i, i, ll, vp, vp, i, i, vp, vp, i, vp, i, ll, vp, sz, vp, vp]
    L.moe_gate_up_i8.argtypes = [vp, vp, i, i, ll, vp, vp, vp, vp, i, i, vp, vp, i, vp, i, ll, vp, sz, vp, vp]
    L.moe_grouped_gemm_i8_expire_wait.argtypes = [vp, vp, i, i, ll, vp, vp, i, i, vp, vp, i, vp, i, ll, vp, sz, vp, i,
                                                  ctypes.c_uint32, vp]
    L.moe_gate_up_i8_expire_wait.argtypes = [vp, vp, i, i, ll, vp, vp, vp, vp, i, i, vp, vp, i, vp, i, ll, vp, sz, vp, i,
                                             ctypes.c_uint32, vp]
    for call in (L.moe_grouped_gemm_i8_expire_wait, L.moe_gate_up_i8_expire_wait, L.moe_dispatch, L.moe_dispatch_filled,
                 L.moe_dispatch_backward, L.moe_combine, L.moe_combine_backward, L.moe_combine_backward_filled, L.moe_quant_i8,
                 L.moe_gemm_i8, L.moe_grouped_gemm_i8, L.moe_gate_up_i8):
        call.restype = i
    L.moe_i8_workspace_size.argtypes = [i, i]
    L.moe_i8_workspace_size.restype = sz
    L.moe_check.argtypes = [vp, vp, vp]
    L.moe_check.restype = i
    L.moe_check_noalloc.argtypes = [vp, vp]
    L.moe_check_noalloc.restype = i
    return L


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _act_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")


def _check(status: int, where: str):
    if status != 0:
        raise MoeError(status, where)


def moe_route(x: torch.Tensor, w_router: torch.Tensor, sel_bias: Optional[torch.Tensor], k: int,
              topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
              scoring: int = MOE_SCORE_SELECTED_SOFTMAX):
    """Router projection + scoring (SelectedSoftmax by default) -> (topk_idx int32
    [T,k], topk_w fp32 [T,k])."""
    L = load_library()
    T, d = x.shape
    E = w_router.shape[0]
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    if scoring == MOE_SCORE_SELECTED_SOFTMAX:
        _check(L.moe_route(_ptr(x), _act_dtype(x), T, d, _ptr(w_router), _ptr(sel_bias), E, k,
                           _ptr(topk_idx), _ptr(topk_w), _stream(x)), "moe_route")
    else:
        _check(L.moe_route_scored(_ptr(x), _act_dtype(x), T, d, _ptr(w_router), _ptr(sel_bias),
                                  E, k, scoring, _ptr(topk_idx), _ptr(topk_w), _stream(x)),
               "moe_route_scored")
    return topk_idx, topk_w


def moe_permute(topk_idx: torch.Tensor, E: int):
    """Token grouping -> (counts [E], offsets [E+1], perm_tok [T*k], inv [T*k]), int32."""
    L = load_library()
    T, k = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm_tok = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    _check(L.moe_permute(_ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm_tok),
                         _ptr(inv), _stream(topk_idx)), "moe_permute")
    return counts, offsets, perm_tok[:T * k], inv[:T * k]


def moe_q8_0_packed_size(rows: int, cols: int) -> int:
    return int(load_library().moe_q8_0_packed_size(rows, cols))


def moe_pack_q8_0(blocks: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Repack Q8_0 blocks (uint8 device tensor, rows*cols/32*34 bytes) into planes."""
    L = load_library()
    n = moe_q8_0_packed_size(rows, cols)
    if n == 0 and rows != 0:
        raise MoeError(1, "moe_q8_0_packed_size")
    packed = torch.empty(max(n, 256), dtype=torch.uint8, device=blocks.device)
    _check(L.moe_pack_q8_0(_ptr(blocks), rows, cols, _ptr(packed), _stream(blocks)),
           "moe_pack_q8_0")
    return packed


def moe_q4_a64_packed_size(rows: int, cols: int) -> int:
    return int(load_library().moe_q4_a64_packed_size(rows, cols))


def moe_pack_q4_a64(blocks: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Repack affine 4-bit group-64 blocks (uint8 device tensor, rows*cols/64*36
    bytes) into the tiles moe_forward takes."""
    L = load_library()
    n = moe_q4_a64_packed_size(rows, cols)
    if n == 0 and rows != 0:
        raise MoeError(1, "moe_q4_a64_packed_size")
    packed = torch.empty(max(n, 256), dtype=torch.uint8, device=blocks.device)
    _check(L.moe_pack_q4_a64(_ptr(blocks), rows, cols, _ptr(packed), _stream(blocks)),
           "moe_pack_q4_a64")
    return packed


def moe_q4_k_packed_size(rows: int, cols: int) -> int:
    return int(load_library().moe_q4_k_packed_size(rows, cols))


def moe_pack_q4_k(blocks: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Repack Q4_K super-blocks (uint8 device tensor, rows*cols/256*144 bytes)
    into the tiles moe_forward takes."""
    L = load_library()
    n = moe_q4_k_packed_size(rows, cols)
    if n == 0 and rows != 0:
        raise MoeError(1, "moe_q4_k_packed_size")
    packed = torch.empty(max(n, 256), dtype=torch.uint8, device=blocks.device)
    _check(L.moe_pack_q4_k(_ptr(blocks), rows, cols, _ptr(packed), _stream(blocks)),
           "moe_pack_q4_k")
    return packed


def moe_q6_k_packed_size(rows: int, cols: int) -> int:
    return int(load_library().moe_q6_k_packed_size(rows, cols))


def moe_pack_q6_k(blocks: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Repack Q6_K super-blocks (uint8 device tensor, rows*cols/256*210 bytes)
    into the 8-bit planes moe_forward takes."""
    L = load_library()
    n = moe_q6_k_packed_size(rows, cols)
    if n == 0 and rows != 0:
        raise MoeError(1, "moe_q6_k_packed_size")
    packed = torch.empty(max(n, 256), dtype=torch.uint8, device=blocks.device)
    _check(L.moe_pack_q6_k(_ptr(blocks), rows, cols, _ptr(packed), _stream(blocks)),
           "moe_pack_q6_k")
    return packed


def moe_fp8_packed_size(rows: int, cols: int) -> int:
    return int(load_library().moe_fp8_packed_size(rows, cols))


def moe_pack_fp8(rows_in: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """Repack fp8 rows {fp32 scale, E4M3 codes} (uint8 device tensor,
    rows*(4+cols) bytes) into the E4M3 plane and row scales moe_forward takes."""
    L = load_library()
    n = moe_fp8_packed_size(rows, cols)
    if n == 0 and rows != 0:
        raise MoeError(1, "moe_fp8_packed_size")
    packed = torch.empty(max(n, 256), dtype=torch.uint8, device=rows_in.device)
    _check(L.moe_pack_fp8(_ptr(rows_in), rows, cols, _ptr(packed), _stream(rows_in)),
           "moe_pack_fp8")
    return packed


def moe_workspace_size(T: int, d: int, E: int, k: int, F: int, act_dt: int, w_dt: int) -> int:
    return int(load_library().moe_workspace_size(T, d, E, k, F, act_dt, w_dt))


def moe_forward(x: torch.Tensor, w_router: torch.Tensor, sel_bias: Optional[torch.Tensor],
                w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, k: int,
                F: Optional[int] = None, w_dtype: Optional[int] = None,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                path: int = MOE_PATH_AUTO, events=None,
                scoring: int = MOE_SCORE_SELECTED_SOFTMAX) -> torch.Tensor:
    """The whole MoE layer -> out fp32 [T, d].

    Weights: float32/bfloat16 tensors [E,F,d], [E,F,d], [E,d,F]; or, with
    w_dtype=MOE_Q8_0 / MOE_Q4_A64 / MOE_Q4_K / MOE_Q6_K / MOE_FP8, uint8 buffers from
    moe_pack_q8_0 / moe_pack_q4_a64 / moe_pack_q4_k / moe_pack_q6_k / moe_pack_fp8 (then F is
    required).
    events: optional sequence of 6 torch.cuda.Event(enable_timing=True), recorded
    at the stage boundaries (moe_forward_profiled).
    scoring: a MOE_SCORE_* mode (moe_forward_scored when not SelectedSoftmax).
    """
    L = load_library()
    T, d = x.shape
    E = w_router.shape[0]
    act = _act_dtype(x)
    if w_dtype is None:
        w_dtype = _act_dtype(w_gate)
    if F is None:
        if w_dtype in PACKED:
            raise ValueError("F is required for block-quantised weights")
        F = w_gate.shape[1]
    if out is None:
        out = torch.empty((T, d), dtype=torch.float32, device=x.device)
    ws_bytes = moe_workspace_size(T, d, E, k, F, act, w_dtype)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=x.device)
    ws_len = workspace.numel() * workspace.element_size()
    if scoring != MOE_SCORE_SELECTED_SOFTMAX:
        handles = None
        if events is not None:
            if len(events) != 6:
                raise ValueError("events: 6 CUDA events expected")
            handles = (ctypes.c_void_p * 6)(*[ev.cuda_event for ev in events])
        _check(L.moe_forward_scored(_ptr(x), act, T, d, _ptr(w_router), _ptr(sel_bias), E, k,
                                    _ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dtype, F,
                                    _ptr(out), _ptr(workspace), ws_len, path, scoring, handles,
                                    _stream(x)), "moe_forward_scored")
    elif events is None:
        _check(L.moe_forward(_ptr(x), act, T, d, _ptr(w_router), _ptr(sel_bias), E, k,
                             _ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dtype, F, _ptr(out),
                             _ptr(workspace), ws_len, path, _stream(x)), "moe_forward")
    else:
        if len(events) != 6:
            raise ValueError("events: 6 CUDA events expected")
        handles = (ctypes.c_void_p * 6)(*[ev.cuda_event for ev in events])
        _check(L.moe_forward_profiled(_ptr(x), act, T, d, _ptr(w_router), _ptr(sel_bias), E, k,
                                      _ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dtype, F,
                                      _ptr(out), _ptr(workspace), ws_len, path, handles,
                                      _stream(x)), "moe_forward_profiled")
    return out


def moe_ffn_dense(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                  w_down: torch.Tensor, F: Optional[int] = None, w_dtype: Optional[int] = None,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  path: int = MOE_PATH_AUTO) -> torch.Tensor:
    """A dense SwiGLU FFN layer -> out fp32 [T, d].

    Weights: float32/bfloat16 tensors [F,d], [F,d], [d,F] (or [1,F,d] ...); or,
    with w_dtype=MOE_Q8_0 / MOE_Q4_A64 / MOE_Q4_K / MOE_Q6_K / MOE_FP8, uint8 buffers from
    moe_pack_q8_0 / moe_pack_q4_a64 / moe_pack_q4_k / moe_pack_q6_k / moe_pack_fp8 (then F is
    required).
    """
    L = load_library()
    T, d = x.shape
    act = _act_dtype(x)
    if w_dtype is None:
        w_dtype = _act_dtype(w_gate)
    if F is None:
        if w_dtype in PACKED:
            raise ValueError("F is required for block-quantised weights")
        F = w_gate.shape[-2]
    if out is None:
        out = torch.empty((T, d), dtype=torch.float32, device=x.device)
    ws_bytes = moe_workspace_size(T, d, 1, 1, F, act, w_dtype)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=x.device)
    ws_len = workspace.numel() * workspace.element_size()
    _check(L.moe_ffn_dense(_ptr(x), act, T, d, _ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dtype, F,
                           _ptr(out), _ptr(workspace), ws_len, path, _stream(x)), "moe_ffn_dense")
    return out


def moe_forward_noalloc(x: torch.Tensor, w_router: torch.Tensor,
                        sel_bias: Optional[torch.Tensor], w_gate: torch.Tensor,
                        w_up: torch.Tensor, w_down: torch.Tensor, k: int, out: torch.Tensor,
                        F: Optional[int] = None, w_dtype: Optional[int] = None,
                        path: int = MOE_PATH_AUTO) -> torch.Tensor:
    """moe_forward without a workspace: the library's static scratch is used.

    For hosts that cannot allocate device memory; `out` must be supplied.
    Layers needing more than 8 MiB of scratch raise MOE_ERR_WORKSPACE.
    """
    L = load_library()
    T, d = x.shape
    E = w_router.shape[0]
    if w_dtype is None:
        w_dtype = _act_dtype(w_gate)
    if F is None:
        if w_dtype in PACKED:
            raise ValueError("F is required for block-quantised weights")
        F = w_gate.shape[1]
    _check(L.moe_forward_noalloc(_ptr(x), _act_dtype(x), T, d, _ptr(w_router), _ptr(sel_bias), E,
                                 k, _ptr(w_gate), _ptr(w_up), _ptr(w_down), w_dtype, F, _ptr(out),
                                 path, _stream(x)), "moe_forward_noalloc")
    return out


VIEW_NAMES = ("topk_idx", "topk_w", "counts", "offsets", "perm_tok", "inv", "perm_w")


def moe_workspace_views(T: int, d: int, E: int, k: int, F: int, act_dt: int, w_dt: int) -> dict:
    """Byte offsets of the routing / grouping arrays a layer call leaves in its
    workspace: {name: offset} for VIEW_NAMES."""
    L = load_library()
    views = (ctypes.c_size_t * 7)()
    _check(L.moe_workspace_views(T, d, E, k, F, act_dt, w_dt, views), "moe_workspace_views")
    return dict(zip(VIEW_NAMES, [int(v) for v in views]))


def read_routing(workspace: torch.Tensor, T: int, d: int, E: int, k: int, F: int, act_dt: int,
                 w_dt: int) -> dict:
    """The routing and grouping a layer call wrote into `workspace` (read after
    the call's stream work completed): views of the workspace bytes, as
    torch tensors on its device."""
    off = moe_workspace_views(T, d, E, k, F, act_dt, w_dt)
    n = T * k
    shapes = {"topk_idx": ((T, k), torch.int32), "topk_w": ((T, k), torch.float32),
              "counts": ((E,), torch.int32), "offsets": ((E + 1,), torch.int32),
              "perm_tok": ((n,), torch.int32), "inv": ((n,), torch.int32),
              "perm_w": ((n,), torch.float32)}
    out = {}
    for name, (shape, dt) in shapes.items():
        count = int(np.prod(shape))
        raw = workspace[off[name]:off[name] + 4 * count]
        out[name] = raw.view(dt).reshape(shape)
    return out


def moe_check_noalloc() -> int:
    """moe_check for moe_forward_noalloc's static scratch on the current device."""
    L = load_library()
    word = ctypes.c_uint32(0)
    _check(L.moe_check_noalloc(ctypes.byref(word), _stream_current()), "moe_check_noalloc")
    return word.value


def _stream_current():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def moe_check(workspace: torch.Tensor) -> int:
    """Wait for the current stream, return the device status word (raises on error)."""
    L = load_library()
    word = ctypes.c_uint32(0)
    _check(L.moe_check(_ptr(workspace), ctypes.byref(word), _stream(workspace)), "moe_check")
    return word.value


# ---- block-scaled fp8 operators (E4M3 codes; one fp32 scale per row and 128
# columns, or per 128 x 128 block).  Their tensors are checked, and their outputs
# allocated, in the compiled module _fp8b (csrc/fp8b_binding.cpp): ValueError /
# TypeError for tensors that do not fit one another, MoeError for what the
# library refuses.

_fp8b_module = None


def _fp8b():
    global _fp8b_module
    if _fp8b_module is None:
        load_library()
        path = _build.binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it for this PyTorch and Python first "
                               "(python -m expert_routed_ffn_selectedsoftmax_gb300.build)")
        spec = importlib.util.spec_from_file_location("_fp8b", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _fp8b_module = module
    return _fp8b_module


def _checked(out, where: str):
    if type(out) is int:   # the status of a refused call
        raise MoeError(out, where)
    return out


def moe_fp8b_workspace_size(rows: int, K: int) -> int:
    return int(load_library().moe_fp8b_workspace_size(rows, K))


def moe_quant_fp8b(x: torch.Tensor, block_rows: int = 1, codes: Optional[torch.Tensor] = None,
                   scales: Optional[torch.Tensor] = None):
    """Block-scaled fp8 of x [rows, cols] or [batch, rows, cols] (fp32 / bf16) ->
    (codes float8_e4m3fn like x, scales fp32 [..., ceil(rows/block_rows), ceil(cols/128)]).

    block_rows: 1 for activations (a scale per row and 128 columns), 128 for
    weights (a scale per 128 x 128 block).
    """
    return _checked((_fp8b_module or _fp8b()).quant(x, block_rows, codes, scales), "moe_quant_fp8b")


def moe_norm_fp8b(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                  delta: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  inv: Optional[torch.Tensor] = None, want_normed: bool = True,
                  resid: Optional[torch.Tensor] = None, normed: Optional[torch.Tensor] = None,
                  codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Residual addition, RMS norm and quantisation -> (resid, normed, codes, scales).

    x [T, d] fp32 / bf16.  delta None: r = x (resid is x itself).  delta [T, d]:
    r = x + delta.  With topk_w [T, k] and inv [T*k] (moe_route, moe_permute):
    delta holds grouped rows, r[t] = x[t] + sum_j topk_w[t, j] delta[inv[t*k + j]].
    resid: r in x's type; normed: bf16 RMS norm of r times weight (None with
    want_normed=False); codes, scales: the same in block-scaled fp8.  resid may
    be x.
    """
    return _checked((_fp8b_module or _fp8b()).norm(x, weight, eps, delta, topk_w, inv, want_normed, resid,
                                                   normed, codes, scales), "moe_norm_fp8b")


def moe_gemm_fp8b(x_q: torch.Tensor, x_s: torch.Tensor, w_q: torch.Tensor, w_s: torch.Tensor,
                  out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                  status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, K] times W^T, W [N, K], in block-scaled fp8 -> out [T, N] bf16 / fp32.

    x_s [T, ceil(K/128)], w_s [ceil(N/128), ceil(K/128)]; x_q's and out's rows
    may be further apart than their length.  status: optional int32 device word
    that collects device-side errors (zero it once; moe_check(status) reads it).
    """
    if w_q.dim() != 2:
        raise ValueError(f"w_q: {w_q.dim()} dimensions, expected 2")
    return _checked((_fp8b_module or _fp8b()).product(x_q, x_s, w_q, w_s, None, None, out, out_dtype, None, status),
                    "moe_gemm_fp8b")


def moe_grouped_gemm_fp8b(x_q: torch.Tensor, x_s: torch.Tensor, w_q: torch.Tensor,
                          w_s: torch.Tensor, offsets: torch.Tensor,
                          perm_tok: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None,
                          out_dtype: torch.dtype = torch.bfloat16,
                          workspace: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every expert's product with its rows, in block-scaled fp8 -> out [rows, N].

    w_q [E, N, K], w_s [E, ceil(N/128), ceil(K/128)]; rows of expert e are
    [offsets[e], offsets[e+1]) (moe_permute), row r is x's row perm_tok[r], or r
    itself without perm_tok.  Rows from offsets[E] on are left as they were.
    workspace: with perm_tok, scratch of moe_fp8b_workspace_size(rows, K) bytes
    (allocated when not given).
    """
    if w_q.dim() != 3:
        raise ValueError(f"w_q: {w_q.dim()} dimensions, expected 3")
    return _checked((_fp8b_module or _fp8b()).product(x_q, x_s, w_q, w_s, offsets, perm_tok, out, out_dtype,
                                                      workspace, status), "moe_grouped_gemm_fp8b")


def moe_gate_up_fp8b(x_q: torch.Tensor, x_s: torch.Tensor, wg_q: torch.Tensor, wg_s: torch.Tensor,
                     wu_q: torch.Tensor, wu_s: torch.Tensor,
                     offsets: Optional[torch.Tensor] = None,
                     perm_tok: Optional[torch.Tensor] = None, h_q: Optional[torch.Tensor] = None,
                     h_s: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None):
    """h = SiLU(W_g x) * (W_u x) per grouped row, quantised -> (h_q [rows, F], h_s).

    wg_q, wu_q [E, F, d] (or [F, d] without offsets: a dense layer) with scales
    [E, ceil(F/128), ceil(d/128)]; offsets, perm_tok and workspace as
    moe_grouped_gemm_fp8b.
    """
    return _checked((_fp8b_module or _fp8b()).gate_up(x_q, x_s, wg_q, wg_s, wu_q, wu_s, offsets, perm_tok, h_q, h_s,
                                                      workspace, status), "moe_gate_up_fp8b")


# ---- rows to their experts and back, and the 8-bit integer operators (int8 codes, one
# fp32 scale per row).  Their tensors are checked, and their outputs allocated, in the
# compiled module too (csrc/i8_binding.cpp).

# Autograd: where an input requires grad and gradients are recorded, the compiled module
# answers NotImplemented, and the call is made by a Function, whose backward pass is made of the
# same four calls (dispatch and its backward are each other's; combine's backward is linear in
# each of grad, y and topk_w).

def _rows(g: torch.Tensor) -> torch.Tensor:
    """A gradient as the calls take it (one of a sum is a single value seen everywhere)."""
    return g if g.stride(1) == 1 and g.stride(0) >= g.shape[1] else g.contiguous()


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, inv, k, rows):
        ctx.save_for_backward(inv)
        ctx.k = k
        if rows is None:
            return moe_dispatch(x, inv, k)
        return moe_dispatch(x, inv, k, out=x.new_zeros(rows, x.shape[1]))

    @staticmethod
    def backward(ctx, g):
        return moe_dispatch_backward(_rows(g), ctx.saved_tensors[0], ctx.k), None, None, None


class _DispatchBackward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad, inv, k):
        ctx.save_for_backward(inv)
        ctx.k, ctx.rows = k, grad.shape[0]
        return moe_dispatch_backward(grad, inv, k)

    @staticmethod
    def backward(ctx, g):
        return _Dispatch.apply(_rows(g), ctx.saved_tensors[0], ctx.k, ctx.rows), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, topk_w, inv, out_dtype):
        ctx.save_for_backward(y, topk_w, inv)
        return moe_combine(y, topk_w, inv, out_dtype=out_dtype)

    @staticmethod
    def backward(ctx, g):
        y, w, inv = ctx.saved_tensors
        return (*moe_combine_backward(_rows(g), y, w, inv, *ctx.needs_input_grad[:2]), None, None)


class _CombineBackward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad, y, topk_w, inv, want_dy, want_dw):
        ctx.save_for_backward(grad, y, topk_w, inv)
        ctx.set_materialize_grads(False)
        return moe_combine_backward(grad, y, topk_w, inv, want_dy, want_dw)

    @staticmethod
    def backward(ctx, of_dy, of_dw):
        grad, y, w, inv = ctx.saved_tensors
        g_grad = g_y = g_w = None
        if of_dy is not None:                     # dy = topk_w grad, by slots
            of_dy = _rows(of_dy)
            if ctx.needs_input_grad[0]:
                g_grad = moe_combine(of_dy, w, inv)
            if ctx.needs_input_grad[2]:
                g_w = moe_combine_backward(grad, of_dy, w, inv, want_dy=False)[1]
        if of_dw is not None:                     # dw = <grad, y>, by slots
            of_dw = of_dw.contiguous()
            if ctx.needs_input_grad[0]:
                more = moe_combine(y, of_dw, inv)
                g_grad = more if g_grad is None else g_grad + more
            if ctx.needs_input_grad[1]:
                g_y = moe_combine_backward(grad, y, of_dw, inv, want_dw=False)[0]
        return None if g_grad is None else g_grad.to(grad.dtype), g_y, g_w, None, None, None


def moe_dispatch(x: torch.Tensor, inv: torch.Tensor, k: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Tokens x [T, d] (fp32 / bf16) into grouped order -> out [rows, d]: out[inv[t*k + j]] = x[t].

    inv [T*k] (moe_permute).  rows is T*k, or out's if it is given.  Rows that no slot
    names are left as they were in an output that is given, and zeros in one allocated
    here; a slot whose inv is outside [0, rows) writes nothing.  Recorded for autograd where x
    requires grad (not into an out that is given: a warning says so).
    """
    got = (_fp8b_module or _fp8b()).dispatch(x, inv, k, out)
    return _Dispatch.apply(x, inv, k, None) if got is NotImplemented else _checked(got, "moe_dispatch")


def moe_dispatch_backward(grad: torch.Tensor, inv: torch.Tensor, k: int,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_dispatch's gradient -> [T, d] in grad's type: out[t] = sum_j grad[inv[t*k + j]].
    Recorded for autograd where grad requires it (not into an out that is given: a warning says so)."""
    got = (_fp8b_module or _fp8b()).dispatch_backward(grad, inv, k, out)
    return _DispatchBackward.apply(grad, inv, k) if got is NotImplemented else _checked(got, "moe_dispatch_backward")


def moe_combine(y: torch.Tensor, topk_w: torch.Tensor, inv: torch.Tensor, out: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The experts' outputs y [rows, d] (fp32 / bf16) back to tokens -> out [T, d] fp32 / bf16:
    out[t] = sum_j topk_w[t, j] y[inv[t*k + j]].

    topk_w [T, k] (moe_route), inv [T*k] (moe_permute); a slot whose inv is outside
    [0, rows) adds nothing.  Recorded for autograd where y or topk_w requires grad (not into
    an out that is given: a warning says so).
    """
    got = (_fp8b_module or _fp8b()).combine(y, topk_w, inv, out, out_dtype)
    return _Combine.apply(y, topk_w, inv, out_dtype) if got is NotImplemented else _checked(got, "moe_combine")


def moe_combine_backward(grad: torch.Tensor, y: torch.Tensor, topk_w: torch.Tensor, inv: torch.Tensor,
                         want_dy: bool = True, want_dw: bool = True, dy: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None):
    """moe_combine's gradients for grad [T, d] -> (dy [rows, d] in y's type, dw fp32 [T, k]):
    dy[inv[t*k + j]] = topk_w[t, j] grad[t], dw[t, j] = <grad[t], y[inv[t*k + j]]>.

    One that is not wanted is None.  Rows of dy that no slot names are left as they were in
    a dy that is given, and zeros (their gradient) in one allocated here.  Recorded for
    autograd where grad, y or topk_w requires it (not into a dy or dw that is given: a warning
    says so).
    """
    got = (_fp8b_module or _fp8b()).combine_backward(grad, y, topk_w, inv, want_dy, want_dw, dy, dw)
    if got is NotImplemented:
        return _CombineBackward.apply(grad, y, topk_w, inv, want_dy, want_dw)
    return _checked(got, "moe_combine_backward")


def moe_i8_workspace_size(rows: int, K: int) -> int:
    return int(load_library().moe_i8_workspace_size(rows, K))


def moe_quant_i8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """int8 codes of x [rows, cols] or [batch, rows, cols] (fp32 / bf16) -> (codes int8 like x,
    scales fp32 [..., rows]): one scale per row, max|x| / 127 (a token of activations, an
    output channel of weights [E, N, K])."""
    return _checked((_fp8b_module or _fp8b()).quant_i8(x, codes, scales), "moe_quant_i8")


def moe_gemm_i8(x_q: torch.Tensor, x_s: torch.Tensor, w_q: torch.Tensor, w_s: torch.Tensor,
                out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [T, K] times W^T, W [N, K], int8 codes with a scale per row of each (x_s [T],
    w_s [N]) -> out [T, N] bf16 / fp32.

    x_q's and out's rows may be further apart than their length.  workspace: scratch of
    moe_i8_workspace_size(T, K) bytes (allocated when not given).  status: optional int32
    device word that collects device-side errors (zero it once; moe_check(status) reads it).
    """
    if w_q.dim() != 2:
        raise ValueError(f"w_q: {w_q.dim()} dimensions, expected 2")
    return _checked((_fp8b_module or _fp8b()).product_i8(x_q, x_s, w_q, w_s, None, None, out, out_dtype, workspace,
                                                         status), "moe_gemm_i8")


def moe_grouped_gemm_i8(x_q: torch.Tensor, x_s: torch.Tensor, w_q: torch.Tensor, w_s: torch.Tensor,
                        offsets: torch.Tensor, perm_tok: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                        workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every expert's product with its rows, int8 codes with a scale per row -> out [rows, N].

    w_q [E, N, K], w_s [E, N]; rows of expert e are [offsets[e], offsets[e+1])
    (moe_permute), row r is x's row perm_tok[r], or r itself without perm_tok.  Rows from
    offsets[E] on are left as they were.  workspace: scratch of
    moe_i8_workspace_size(rows, K) bytes (allocated when not given).
    """
    if w_q.dim() != 3:
        raise ValueError(f"w_q: {w_q.dim()} dimensions, expected 3")
    return _checked((_fp8b_module or _fp8b()).product_i8(x_q, x_s, w_q, w_s, offsets, perm_tok, out, out_dtype,
                                                         workspace, status), "moe_grouped_gemm_i8")


def moe_gate_up_i8(x_q: torch.Tensor, x_s: torch.Tensor, wg_q: torch.Tensor, wg_s: torch.Tensor,
                   wu_q: torch.Tensor, wu_s: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                   perm_tok: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                   h_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h = SiLU(W_g x) * (W_u x) per grouped row -> h [rows, F] bf16 / fp32.

    wg_q, wu_q [E, F, d] (or [F, d] without offsets: a dense layer) with scales [E, F];
    offsets, perm_tok and workspace as moe_grouped_gemm_i8.  moe_quant_i8(h) gives the down
    projection's codes.
    """
    return _checked((_fp8b_module or _fp8b()).gate_up_i8(x_q, x_s, wg_q, wg_s, wu_q, wu_s, offsets, perm_tok, h, h_dtype,
                                                         workspace, status), "moe_gate_up_i8")
