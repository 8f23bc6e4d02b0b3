"""Python binding of libsp24 (the C ABI declared in include/sp24.h).

Argument marshalling only: every step of the pipeline runs in the CUDA kernels of
``libsp24.so``.  PyTorch supplies device memory and the current stream.  There is no CPU path:
the functions accept CUDA tensors only and raise when the library cannot be loaded.

Pipeline ([P1] "NVFP4 vs 2:4 sparse: where the other half of the petaflop went",
[P2] "Sparse GPU FLOPS Need the Right Zeros in the Right Places", [P5] "NVFP4 Without FP4
Hardware"):

    check_24 -> prune_compress_24 -> quantize_nvfp4 -> gemm_dense / gemm_sparse24

Routed feed-forward around gemm_grouped / moe_block, and its single-token form with 4-bit weights:

    moe_route -> moe_sort -> gemm_grouped or gemv_w4_grouped -> moe_unsort, each with its _backward
    (moe_sort_backward, moe_unsort_backward, moe_route_backward) where it is differentiable

No entry point records anything for autograd: outputs are detached, also where inputs require
gradients.  The products (gemm_*, gemv_w4*, moe_block) have no gradient here.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsp24.so")

# status codes (include/sp24.h)
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_CUDA, \
    ERR_DEVICE_TIMEOUT, ERR_WORKSPACE = range(9)
F16, BF16, F32, NVFP4, NVFP4_B32, NVFP4_MMA, NVFP4_B32_MMA = 0, 1, 2, 3, 4, 5, 6
OP_MATMUL, OP_CONV = 0, 1
ALGO_AUTO, ALGO_SKINNY, ALGO_TILED = 0, 1, 2
ROUTE_SOFTMAX, ROUTE_SIGMOID = 0, 1
ACT_NONE, ACT_SWIGLU = 0, 1

EXPORTS = ("sp24_status_string", "sp24_abi_version", "sp24_sizes", "sp24_check_24",
           "sp24_prune_compress_24", "sp24_decompress_24", "sp24_quantize_nvfp4_workspace_size",
           "sp24_quantize_nvfp4", "sp24_dequantize_nvfp4", "sp24_gemm_workspace_size",
           "sp24_gemm_dense", "sp24_gemm_sparse24", "sp24_kernel_launches",
           "sp24_last_device_error", "sp24_quantize_nvfp4_noalloc", "sp24_gemm_grouped_workspace_size",
           "sp24_gemm_grouped", "sp24_prepare_24_workspace_size", "sp24_prepare_24",
           "sp24_quantize_nvfp4_pair", "sp24_nvfp4_group_tensor_scale_workspace_size",
           "sp24_nvfp4_group_tensor_scale", "sp24_gemm_select", "sp24_gemm_choice", "sp24_gemm_auto",
           "sp24_gemm_choice_reset", "sp24_moe_block_workspace_size", "sp24_moe_block",
           "sp24_interleave_rows", "sp24_check_48", "sp24_prune_compress_48", "sp24_decompress_48",
           "sp24_quantize_nvfp4_block32", "sp24_gemm_sparse48", "sp24_moe_route", "sp24_moe_route_backward",
           "sp24_moe_sort_workspace_size", "sp24_moe_sort", "sp24_moe_unsort", "sp24_moe_unsort_backward",
           "sp24_quantize_w4", "sp24_dequantize_w4", "sp24_gemv_w4", "sp24_gemv_w4_grouped")

_lock = threading.Lock()
_lib = None


class SP24Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.sp24_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


class _Operand(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("data", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p)]


class _SparseOperand(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("values", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("meta", ctypes.c_void_p)]


class _W4Operand(ctypes.Structure):
    _fields_ = [("scale_dtype", ctypes.c_int32), ("group", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    """Loads libsp24.so (building it in-tree first if it is missing or older than a source)."""
    global _lib
    with _lock:
        if _lib is None:
            from . import build as _build
            if _build.stale():
                _build.build()
            L = ctypes.CDLL(LIB_PATH)
            P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
            L.sp24_status_string.restype = ctypes.c_char_p
            L.sp24_status_string.argtypes = [I]
            L.sp24_sizes.argtypes = [I, I, P, I, P, P, P, P, P]
            L.sp24_check_24.argtypes = [P, I, I, P, I, P, P, P]
            L.sp24_prune_compress_24.argtypes = [P, I, I, P, I, P, P, P]
            L.sp24_decompress_24.argtypes = [P, P, I, I, P, I, P, P]
            L.sp24_quantize_nvfp4_workspace_size.argtypes = [I64, I64, P]
            L.sp24_quantize_nvfp4.argtypes = [P, I, I64, I64, P, P, P, P, P, I64, P]
            L.sp24_dequantize_nvfp4.argtypes = [P, P, P, I64, I64, I, P, P]
            L.sp24_quantize_nvfp4_noalloc.argtypes = [P, I, I64, I64, P, P, P, P, P]
            L.sp24_gemm_workspace_size.argtypes = [I, I, I, I64, I64, I64, I, P]
            L.sp24_gemm_dense.argtypes = [ctypes.POINTER(_Operand), ctypes.POINTER(_Operand), I64,
                                          I64, I64, P, P, I64, I, P]
            L.sp24_gemm_sparse24.argtypes = [ctypes.POINTER(_Operand),
                                             ctypes.POINTER(_SparseOperand), I64, I64, I64, P, P,
                                             I64, I, P]
            L.sp24_last_device_error.argtypes = [P]
            L.sp24_gemm_grouped_workspace_size.argtypes = [I64, I, I64, P]
            L.sp24_gemm_grouped.argtypes = [ctypes.POINTER(_Operand), P, I64, I, ctypes.POINTER(_Operand),
                                             ctypes.POINTER(_SparseOperand), I64, I64, I64, P, P, I64, P]
            L.sp24_prepare_24_workspace_size.argtypes = [I64, I64, P]
            L.sp24_prepare_24.argtypes = [P, I, I64, I64, P, P, P, P, P, P, P, I64, P]
            L.sp24_quantize_nvfp4_pair.argtypes = [P, I, I64, I64, P, P, P, P, P, I64, I64, P, P, P, P, P]
            L.sp24_nvfp4_group_tensor_scale_workspace_size.argtypes = [P]
            L.sp24_nvfp4_group_tensor_scale.argtypes = [P, P, I, I, P, P, I64, P]
            L.sp24_gemm_select.argtypes = [ctypes.POINTER(_Operand), ctypes.POINTER(_Operand),
                                           ctypes.POINTER(_SparseOperand), I64, I64, I64, P, P, I64, I,
                                           P, P, P, P]
            L.sp24_gemm_choice.argtypes = [I, I, I64, I64, I64, P, P]
            L.sp24_gemm_auto.argtypes = [ctypes.POINTER(_Operand), ctypes.POINTER(_Operand),
                                         ctypes.POINTER(_SparseOperand), I64, I64, I64, P, P, I64, P, P]
            L.sp24_gemm_choice_reset.argtypes = []
            L.sp24_moe_block_workspace_size.argtypes = [I64, I, I64, I64, I64, P]
            L.sp24_moe_block.argtypes = [ctypes.POINTER(_Operand), P, P, I64, I, ctypes.POINTER(_Operand),
                                         ctypes.POINTER(_SparseOperand), ctypes.POINTER(_Operand),
                                         ctypes.POINTER(_SparseOperand), I64, I64, I64, P, P, I64, P]
            L.sp24_interleave_rows.argtypes = [P, P, I64, I64, I64, P, P]
            L.sp24_check_48.argtypes = [P, I, I64, I64, P, P, P]
            L.sp24_prune_compress_48.argtypes = [P, I, I64, I64, P, P, P]
            L.sp24_decompress_48.argtypes = [P, P, I, I64, I64, P, P]
            L.sp24_quantize_nvfp4_block32.argtypes = [P, I, I64, I64, P, P, P, P, P, I64, P]
            L.sp24_gemm_sparse48.argtypes = [ctypes.POINTER(_Operand), ctypes.POINTER(_SparseOperand), I64, I64,
                                             I64, P, P]
            L.sp24_nvfp4_mma_size.argtypes = [I64, I64, P, P]
            L.sp24_nvfp4_to_mma.argtypes = [P, P, I64, I64, P, P, P]
            L.sp24_set_wait_limit.argtypes = [ctypes.c_ulonglong]
            L.sp24_get_wait_limit.argtypes = [P]
            L.sp24_selftest_wait_timeout.argtypes = [P, P, P]
            L.sp24_nvfp4_b32_mma_size.argtypes = [I64, I64, P, P]
            L.sp24_nvfp4_b32_to_mma.argtypes = [P, P, I64, I64, P, P, P]
            L.sp24_sparse48_mma_size.argtypes = [I64, I64, P, P, P]
            L.sp24_prepare_sparse_size.argtypes = [I64, I64, P]
            L.sp24_prepare_sparse.argtypes = [P, I64, I64, P, P]
            L.sp24_sparse48_to_mma.argtypes = [P, P, P, I64, I64, P, P, P, P]
            W4 = P  # a _W4Operand by reference, or its bytes
            L.sp24_moe_route.argtypes = [P, I, I64, I64, I, I, I, P, P, P]
            L.sp24_moe_route_backward.argtypes = [P, I, P, P, I64, I64, I, I, I, P, P]
            L.sp24_moe_sort_workspace_size.argtypes = [I64, I, I64, P]
            L.sp24_moe_sort.argtypes = [P, I, P, I64, I, I64, I64, P, P, P, P, P, P, I64, P]
            L.sp24_moe_unsort.argtypes = [P, I, P, P, I64, I, I64, I64, P, I, P]
            L.sp24_moe_unsort_backward.argtypes = [P, I, P, I, P, P, I64, I, I64, I64, P, P, P]
            L.sp24_quantize_w4.argtypes = [P, I, I64, I64, I, I, P, P, P, P]
            L.sp24_dequantize_w4.argtypes = [W4, I64, I64, I, P, P]
            L.sp24_gemv_w4.argtypes = [P, I, W4, I64, I64, I64, I, P, I, P]
            L.sp24_gemv_w4_grouped.argtypes = [P, I, W4, P, I64, I64, I64, I64, I, P, I, P]
            L.sp24_peak_mma.argtypes = [I, I, P, P]
            L.sp24_peak_ctas.argtypes = [I]
            L.sp24_peak_read.argtypes = [P, I64, P, P]
            L.sp24_kernel_launches.restype = I64
            L.sp24_kernel_launches.argtypes = []
            _lib = L
    return _lib


# ---------------------------------------------------------------------------- marshalling

_DT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_TORCH = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _shape(shape) -> ctypes.Array:
    arr = (ctypes.c_int64 * 4)()
    for i, s in enumerate(shape):
        arr[i] = int(s)
    return arr


def _call(fn: str, *args) -> None:
    st = getattr(lib(), fn)(*args)
    if st != OK:
        raise SP24Error(st, fn)


def _groups(op: int, shape) -> int:
    shape = tuple(int(s) for s in shape)
    if op == OP_MATMUL:
        n = 1
        for s in shape:
            n *= s
        return n // 4
    K, C, R, S = shape
    return K * (C // 4) * R * S


def group_shape(op: int, shape) -> tuple:
    shape = tuple(int(s) for s in shape)
    if op == OP_MATMUL:
        return shape[:-1] + (shape[-1] // 4,)
    K, C, R, S = shape
    return (K, C // 4, R, S)


def values_shape(op: int, shape) -> tuple:
    shape = tuple(int(s) for s in shape)
    if op == OP_MATMUL:
        return shape[:-1] + (shape[-1] // 2,)
    K, C, R, S = shape
    return (K, C // 2, R, S)


class NVFP4Tensor(NamedTuple):
    """codes uint8 [rows, cols/2], scales uint8 [rows, cols/16], tensor_scale fp32 [1]."""
    codes: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor


class NVFP4MMA(NamedTuple):
    """An NVFP4 tensor as the W4A4 GEMM's tile images (see to_mma): codes and scales are flat
    uint8 tensors (rows padded to a multiple of 128), tensor_scale fp32 [1]; rows, cols the
    logical shape."""
    codes: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor
    rows: int
    cols: int


class Sparse24(NamedTuple):
    """A 2:4-compressed weight [N, K]: values ([N, K/2] 16-bit, or NVFP4 of them) + meta."""
    values: object  # torch.Tensor (16-bit) or NVFP4Tensor
    meta: torch.Tensor


# ---------------------------------------------------------------------------- a1 .. a3

def check_24(w: torch.Tensor, op: int = OP_MATMUL, pass_out=None, n_fail_out=None, stream=None):
    """Per-group eligibility (uint8 0/1) and the failing-group count (int32 [1], device)."""
    _cuda(w, "w")
    if pass_out is None:
        pass_out = torch.empty(group_shape(op, w.shape), dtype=torch.uint8, device=w.device)
    if n_fail_out is None:
        n_fail_out = torch.empty(1, dtype=torch.int32, device=w.device)
    _call("sp24_check_24", _ptr(w), _dtype_code(w), op, _shape(w.shape), w.dim(),
          _ptr(pass_out), _ptr(n_fail_out), _stream(stream))
    return pass_out, n_fail_out


def prune_compress_24(w: torch.Tensor, op: int = OP_MATMUL, values_out=None, meta_out=None,
                      stream=None):
    """(values, meta): kept entries [.., K/2] (or [K, C/2, R, S]) and the nibble stream."""
    _cuda(w, "w")
    if values_out is None:
        values_out = torch.empty(values_shape(op, w.shape), dtype=w.dtype, device=w.device)
    if meta_out is None:
        meta_out = torch.empty((_groups(op, w.shape) + 1) // 2, dtype=torch.uint8, device=w.device)
    _call("sp24_prune_compress_24", _ptr(w), _dtype_code(w), op, _shape(w.shape), w.dim(),
          _ptr(values_out), _ptr(meta_out), _stream(stream))
    return values_out, meta_out


def decompress_24(values: torch.Tensor, meta: torch.Tensor, shape, op: int = OP_MATMUL,
                  out=None, stream=None):
    _cuda(values, "values")
    _cuda(meta, "meta")
    if out is None:
        out = torch.empty(tuple(shape), dtype=values.dtype, device=values.device)
    _call("sp24_decompress_24", _ptr(values), _ptr(meta), _dtype_code(values), op, _shape(shape),
          len(shape), _ptr(out), _stream(stream))
    return out


def _rows_k48(shape) -> tuple:
    shape = tuple(int(d) for d in shape)
    if not shape:
        raise ValueError("pairwise 4:8 needs at least one axis")
    K = shape[-1]
    rows = 1
    for d in shape[:-1]:
        rows *= d
    return rows, K


def check_48(w: torch.Tensor, pass_out=None, n_fail_out=None, stream=None):
    """Pairwise 4:8 eligibility per chunk of 8 along K (uint8 0/1, [.., K/8]) and the failing
    chunk count (int32 [1], device)."""
    _cuda(w, "w")
    rows, K = _rows_k48(w.shape)
    if pass_out is None:
        pass_out = torch.empty(tuple(w.shape[:-1]) + (K // 8,), dtype=torch.uint8, device=w.device)
    if n_fail_out is None:
        n_fail_out = torch.empty(1, dtype=torch.int32, device=w.device)
    _call("sp24_check_48", _ptr(w), _dtype_code(w), rows, K, _ptr(pass_out), _ptr(n_fail_out), _stream(stream))
    return pass_out, n_fail_out


def prune_compress_48(w: torch.Tensor, values_out=None, meta_out=None, stream=None):
    """(values [.., K/2], meta): the two kept pairs of every chunk of 8 and the nibble stream."""
    _cuda(w, "w")
    rows, K = _rows_k48(w.shape)
    if values_out is None:
        values_out = torch.empty(tuple(w.shape[:-1]) + (K // 2,), dtype=w.dtype, device=w.device)
    if meta_out is None:
        meta_out = torch.empty((rows * (K // 8) + 1) // 2, dtype=torch.uint8, device=w.device)
    _call("sp24_prune_compress_48", _ptr(w), _dtype_code(w), rows, K, _ptr(values_out), _ptr(meta_out),
          _stream(stream))
    return values_out, meta_out


def decompress_48(values: torch.Tensor, meta: torch.Tensor, shape, out=None, stream=None):
    _cuda(values, "values")
    _cuda(meta, "meta")
    rows, K = _rows_k48(shape)
    if out is None:
        out = torch.empty(tuple(shape), dtype=values.dtype, device=values.device)
    _call("sp24_decompress_48", _ptr(values), _ptr(meta), _dtype_code(values), rows, K, _ptr(out),
          _stream(stream))
    return out


def quantize_workspace_bytes(rows: int, cols: int) -> int:
    n = ctypes.c_int64(0)
    _call("sp24_quantize_nvfp4_workspace_size", rows, cols, ctypes.byref(n))
    return n.value


def quantize_nvfp4(t: torch.Tensor, tensor_scale: Optional[torch.Tensor] = None, out=None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> NVFP4Tensor:
    """NVFP4 of a 2-D tensor; `tensor_scale` (fp32 [1], device) shares a scale across tensors."""
    _cuda(t, "t")
    if t.dim() != 2:
        raise ValueError("quantize_nvfp4 wants a 2-D tensor")
    R, L = t.shape
    if out is None:
        out = NVFP4Tensor(torch.empty((R, L // 2), dtype=torch.uint8, device=t.device),
                          torch.empty((R, L // 16), dtype=torch.uint8, device=t.device),
                          torch.empty(1, dtype=torch.float32, device=t.device))
    if workspace is None and tensor_scale is None:
        workspace = torch.empty(quantize_workspace_bytes(R, L), dtype=torch.uint8, device=t.device)
    _call("sp24_quantize_nvfp4", _ptr(t), _dtype_code(t), R, L, _ptr(tensor_scale),
          _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), _ptr(workspace),
          0 if workspace is None else workspace.numel(), _stream(stream))
    return out


def quantize_nvfp4_block32(t: torch.Tensor, tensor_scale: Optional[torch.Tensor] = None, out=None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> NVFP4Tensor:
    """E2M1 codes with one E4M3 scale per 32 entries (scales [R, L/32]): the activation form of
    the pairwise-4:8 FP4 GEMM (gemm_sparse48)."""
    _cuda(t, "t")
    if t.dim() != 2:
        raise ValueError("quantize_nvfp4_block32 wants a 2-D tensor")
    R, L = t.shape
    if out is None:
        out = NVFP4Tensor(torch.empty((R, L // 2), dtype=torch.uint8, device=t.device),
                          torch.empty((R, L // 32), dtype=torch.uint8, device=t.device),
                          torch.empty(1, dtype=torch.float32, device=t.device))
    if workspace is None and tensor_scale is None:
        workspace = torch.empty(quantize_workspace_bytes(R, L), dtype=torch.uint8, device=t.device)
    _call("sp24_quantize_nvfp4_block32", _ptr(t), _dtype_code(t), R, L, _ptr(tensor_scale),
          _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), _ptr(workspace),
          0 if workspace is None else workspace.numel(), _stream(stream))
    return out


def nvfp4_group_tensor_scale(tensors, out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One NVFP4 tensor scale (fp32 [1], device) shared by a group of tensors of one dtype:
    max amax / 2688 over all of them.  Pass it to quantize_nvfp4(t, tensor_scale=...)."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("nvfp4_group_tensor_scale wants at least one tensor")
    for i, t in enumerate(tensors):
        _cuda(t, f"tensors[{i}]")
        if not t.is_contiguous() or t.dtype != tensors[0].dtype:
            raise ValueError("nvfp4_group_tensor_scale wants contiguous tensors of one dtype")
    dev = tensors[0].device
    if out is None:
        out = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        nb = ctypes.c_int64(0)
        _call("sp24_nvfp4_group_tensor_scale_workspace_size", ctypes.byref(nb))
        workspace = torch.empty(nb.value, dtype=torch.uint8, device=dev)
    n = len(tensors)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors])
    numels = (ctypes.c_int64 * n)(*[t.numel() for t in tensors])
    _call("sp24_nvfp4_group_tensor_scale", ptrs, numels, n, _dtype_code(tensors[0]), _ptr(out),
          _ptr(workspace), workspace.numel(), _stream(stream))
    return out


def quantize_nvfp4_pair(t0: torch.Tensor, ts0: torch.Tensor, t1: torch.Tensor, ts1: torch.Tensor,
                        out0=None, out1=None, stream=None):
    """NVFP4 of two 2-D tensors of one dtype in one launch, each with its supplied tensor scale
    (fp32 [1], device); identical to quantize_nvfp4(t0, ts0) and quantize_nvfp4(t1, ts1)."""
    _cuda(t0, "t0")
    _cuda(t1, "t1")
    if t0.dim() != 2 or t1.dim() != 2 or t0.dtype != t1.dtype:
        raise ValueError("quantize_nvfp4_pair wants two 2-D tensors of one dtype")
    outs = []
    for t, o in ((t0, out0), (t1, out1)):
        R, L = t.shape
        outs.append(o if o is not None else NVFP4Tensor(
            torch.empty((R, L // 2), dtype=torch.uint8, device=t.device),
            torch.empty((R, L // 16), dtype=torch.uint8, device=t.device),
            torch.empty(1, dtype=torch.float32, device=t.device)))
    a, b = outs
    _call("sp24_quantize_nvfp4_pair", _ptr(t0), _dtype_code(t0), t0.shape[0], t0.shape[1], _ptr(ts0),
          _ptr(a.codes), _ptr(a.scales), _ptr(a.tensor_scale), _ptr(t1), t1.shape[0], t1.shape[1],
          _ptr(ts1), _ptr(b.codes), _ptr(b.scales), _ptr(b.tensor_scale), _stream(stream))
    return a, b


def quantize_nvfp4_noalloc(t: torch.Tensor, tensor_scale: Optional[torch.Tensor] = None, out=None,
                           stream=None) -> NVFP4Tensor:
    """quantize_nvfp4 without a workspace: the library's own per-device scratch is used, so the
    call needs no device allocation (for callers that cannot allocate, e.g. during graph
    capture).  Calls whose GPU work overlaps race on that scratch."""
    _cuda(t, "t")
    if t.dim() != 2:
        raise ValueError("quantize_nvfp4_noalloc wants a 2-D tensor")
    R, L = t.shape
    if out is None:
        out = NVFP4Tensor(torch.empty((R, L // 2), dtype=torch.uint8, device=t.device),
                          torch.empty((R, L // 16), dtype=torch.uint8, device=t.device),
                          torch.empty(1, dtype=torch.float32, device=t.device))
    _call("sp24_quantize_nvfp4_noalloc", _ptr(t), _dtype_code(t), R, L, _ptr(tensor_scale),
          _ptr(out.codes), _ptr(out.scales), _ptr(out.tensor_scale), _stream(stream))
    return out


def dequantize_nvfp4(q: NVFP4Tensor, dtype=torch.float32, stream=None) -> torch.Tensor:
    R, L2 = q.codes.shape
    out = torch.empty((R, 2 * L2), dtype=dtype, device=q.codes.device)
    _call("sp24_dequantize_nvfp4", _ptr(q.codes), _ptr(q.scales), _ptr(q.tensor_scale), R, 2 * L2,
          _DT[dtype], _ptr(out), _stream(stream))
    return out


class Prepared24(NamedTuple):
    """What sp24_prepare_24 produces for a weight W[rows, K]."""
    pass_map: Optional[torch.Tensor]   # uint8 [rows, K/4] or None
    n_fail: torch.Tensor               # int32 [1]
    values: torch.Tensor               # kept entries [rows, K/2], W's dtype
    meta: torch.Tensor                 # uint8 [rows, K/8] nibble stream
    w_tensor_scale: torch.Tensor       # fp32 [1]: amax|W| / 2688
    v_tensor_scale: torch.Tensor       # fp32 [1]: amax|values| / 2688


def prepare_workspace_bytes(rows: int, K: int) -> int:
    n = ctypes.c_int64(0)
    _call("sp24_prepare_24_workspace_size", rows, K, ctypes.byref(n))
    return n.value


def prepare_24(w: torch.Tensor, with_pass: bool = True, out: Optional[Prepared24] = None,
               workspace=None, stream=None) -> Prepared24:
    """check_24 + prune_compress_24 + both NVFP4 tensor scales of a matmul weight w[rows, K]
    (K % 16 == 0) with one read of w; identical to the separate calls."""
    _cuda(w, "w")
    if w.dim() != 2:
        raise ValueError("prepare_24 wants a 2-D weight")
    R, K = w.shape
    dev = w.device
    if out is None:
        out = Prepared24(
            torch.empty((R, K // 4), dtype=torch.uint8, device=dev) if with_pass else None,
            torch.empty(1, dtype=torch.int32, device=dev),
            torch.empty((R, K // 2), dtype=w.dtype, device=dev),
            torch.empty((R, K // 8), dtype=torch.uint8, device=dev),
            torch.empty(1, dtype=torch.float32, device=dev),
            torch.empty(1, dtype=torch.float32, device=dev))
    if workspace is None:
        workspace = torch.empty(prepare_workspace_bytes(R, K), dtype=torch.uint8, device=dev)
    _call("sp24_prepare_24", _ptr(w), _dtype_code(w), R, K, _ptr(out.pass_map), _ptr(out.n_fail),
          _ptr(out.values), _ptr(out.meta), _ptr(out.w_tensor_scale), _ptr(out.v_tensor_scale),
          _ptr(workspace), workspace.numel(), _stream(stream))
    return out


def prepare_nvfp4_24(w: torch.Tensor, stream=None):
    """The whole weight side of both GEMM paths: prepare_24, then NVFP4 of w and of its kept
    values with the tensor scales prepare_24 derived.  Returns (Prepared24, dense NVFP4Tensor,
    Sparse24 with NVFP4 values)."""
    p = prepare_24(w, stream=stream)
    wq, vq = quantize_nvfp4_pair(w, p.w_tensor_scale, p.values, p.v_tensor_scale, stream=stream)
    return p, wq, Sparse24(vq, p.meta)


# ---------------------------------------------------------------------------- a4 .. a6

def to_mma(q: NVFP4Tensor, stream=None) -> NVFP4MMA:
    """The same NVFP4 tensor rewritten as the tile images the W4A4 GEMM loads whole
    (sp24_nvfp4_to_mma; cols % 256 == 0); the tensor scale is shared, not copied."""
    rows, cols = q.codes.shape[0], 2 * q.codes.shape[1]
    nc, ns = ctypes.c_int64(0), ctypes.c_int64(0)
    _call("sp24_nvfp4_mma_size", rows, cols, ctypes.byref(nc), ctypes.byref(ns))
    codes = torch.empty(nc.value, dtype=torch.uint8, device=q.codes.device)
    scales = torch.empty(ns.value, dtype=torch.uint8, device=q.codes.device)
    _call("sp24_nvfp4_to_mma", _ptr(q.codes), _ptr(q.scales), rows, cols, _ptr(codes), _ptr(scales),
          _stream(stream))
    return NVFP4MMA(codes, scales, q.tensor_scale, rows, cols)


def _operand(t) -> _Operand:
    if isinstance(t, NVFP4Tensor):
        return _Operand(NVFP4, t.codes.data_ptr(), t.scales.data_ptr(), t.tensor_scale.data_ptr())
    if isinstance(t, NVFP4MMA):
        return _Operand(NVFP4_MMA, t.codes.data_ptr(), t.scales.data_ptr(), t.tensor_scale.data_ptr())
    _cuda(t, "operand")
    return _Operand(_dtype_code(t), t.data_ptr(), None, None)


def _rows_k(t) -> tuple:
    if isinstance(t, NVFP4MMA):
        return t.rows, t.cols
    if isinstance(t, NVFP4Tensor):
        return t.codes.shape[0], 2 * t.codes.shape[1]
    return t.shape[0], t.shape[1]


def gemm_workspace_bytes(x, w, sparse: bool, M: int, N: int, K: int, algo: int = ALGO_AUTO) -> int:
    fmt = lambda t: NVFP4 if isinstance(t, NVFP4Tensor) else NVFP4_MMA if isinstance(t, NVFP4MMA) else _DT[t.dtype]
    xf = fmt(x)
    wf = fmt(w.values if sparse else w)
    n = ctypes.c_int64(0)
    _call("sp24_gemm_workspace_size", xf, wf, int(sparse), M, N, K, algo, ctypes.byref(n))
    return n.value


def gemm_dense(x, w, out=None, algo: int = ALGO_AUTO, workspace=None, stream=None) -> torch.Tensor:
    """Y[M, N] fp32 = x[M, K] @ w[N, K]^T; x, w: 16-bit tensors or NVFP4Tensor."""
    M, K = _rows_k(x)
    N, Kw = _rows_k(w)
    if K != Kw:
        raise ValueError(f"K mismatch: {K} vs {Kw}")
    dev = (x.codes if isinstance(x, (NVFP4Tensor, NVFP4MMA)) else x).device
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    ws_bytes = gemm_workspace_bytes(x, w, False, M, N, K, algo)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    xo, wo = _operand(x), _operand(w)
    _call("sp24_gemm_dense", ctypes.byref(xo), ctypes.byref(wo), M, N, K, _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), algo, _stream(stream))
    return out


def gemm_sparse24(x, w: Sparse24, K: int, out=None, algo: int = ALGO_AUTO, workspace=None,
                  stream=None) -> torch.Tensor:
    """The same product with w 2:4-compressed (values 16-bit or NVFP4 + meta)."""
    M, Kx = _rows_k(x)
    if Kx != K:
        raise ValueError(f"K mismatch: {Kx} vs {K}")
    v = w.values
    if isinstance(v, NVFP4Tensor):
        N = v.codes.shape[0]
        wo = _SparseOperand(NVFP4, v.codes.data_ptr(), v.scales.data_ptr(),
                            v.tensor_scale.data_ptr(), w.meta.data_ptr())
    else:
        _cuda(v, "values")
        N = v.shape[0]
        wo = _SparseOperand(_dtype_code(v), v.data_ptr(), None, None, w.meta.data_ptr())
    dev = w.meta.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    ws_bytes = gemm_workspace_bytes(x, w, True, M, N, K, algo)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    xo = _operand(x)
    _call("sp24_gemm_sparse24", ctypes.byref(xo), ctypes.byref(wo), M, N, K, _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), algo, _stream(stream))
    return out


class Sparse48(NamedTuple):
    """A pairwise-4:8 weight [N, K] for the sparse FP4 MMA: the kept values [N, K/2] as NVFP4
    (16-value blocks: codes [N, K/4], scales [N, K/32]) + the nibble stream of prune_compress_48."""
    values: NVFP4Tensor
    meta: torch.Tensor


class Sparse48MMA(NamedTuple):
    """A pairwise-4:8 weight [rows, K] as the sparse FP4 pair kernel's tile images (flat uint8:
    values, scales, metadata; rows padded to 256), with its tensor scale."""
    values: torch.Tensor
    scales: torch.Tensor
    meta: torch.Tensor
    tensor_scale: torch.Tensor
    rows: int
    K: int


def sparse48_to_mma(w: Sparse48, K: int, stream=None) -> Sparse48MMA:
    """The weight rewritten as tile images (sp24_sparse48_to_mma), once per weight."""
    v = w.values
    rows = v.codes.shape[0]
    nv, ns, nm = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
    _call("sp24_sparse48_mma_size", rows, K, ctypes.byref(nv), ctypes.byref(ns), ctypes.byref(nm))
    dev = v.codes.device
    vo = torch.empty(nv.value, dtype=torch.uint8, device=dev)
    so = torch.empty(ns.value, dtype=torch.uint8, device=dev)
    mo = torch.empty(nm.value, dtype=torch.uint8, device=dev)
    _call("sp24_sparse48_to_mma", _ptr(v.codes), _ptr(v.scales), _ptr(w.meta), rows, K, _ptr(vo), _ptr(so), _ptr(mo),
          _stream(stream))
    return Sparse48MMA(vo, so, mo, v.tensor_scale, rows, K)


def prepare_sparse(meta: torch.Tensor, rows: int, K: int, stream=None) -> torch.Tensor:
    """The 2:4 nibble stream of a [rows, K] weight in the tensor cores' metadata layout
    (sp24_prepare_sparse): uint8 tiles of 2 KB per 128 rows and 128 K, rows padded to 256."""
    n = ctypes.c_int64(0)
    _call("sp24_prepare_sparse_size", rows, K, ctypes.byref(n))
    out = torch.empty(n.value, dtype=torch.uint8, device=meta.device)
    _call("sp24_prepare_sparse", _ptr(meta), rows, K, _ptr(out), _stream(stream))
    return out


def b32_to_mma(q: NVFP4Tensor, stream=None) -> NVFP4MMA:
    """Activations from quantize_nvfp4_block32 rewritten as tile images (sp24_nvfp4_b32_to_mma)."""
    rows, cols = q.codes.shape[0], 2 * q.codes.shape[1]
    nc, ns = ctypes.c_int64(0), ctypes.c_int64(0)
    _call("sp24_nvfp4_b32_mma_size", rows, cols, ctypes.byref(nc), ctypes.byref(ns))
    codes = torch.empty(nc.value, dtype=torch.uint8, device=q.codes.device)
    scales = torch.empty(ns.value, dtype=torch.uint8, device=q.codes.device)
    _call("sp24_nvfp4_b32_to_mma", _ptr(q.codes), _ptr(q.scales), rows, cols, _ptr(codes), _ptr(scales),
          _stream(stream))
    return NVFP4MMA(codes, scales, q.tensor_scale, rows, cols)


def gemm_sparse48(x, w, K: int, out=None, stream=None) -> torch.Tensor:
    """y[M, N] = x w^T on the sparse FP4 MMA: x from quantize_nvfp4_block32 ([M, K]), w a
    pairwise-4:8 weight; K % 512 == 0.  With both operands as tile images (b32_to_mma,
    sparse48_to_mma) the persistent CTA-pair kernel runs."""
    if isinstance(x, NVFP4MMA) or isinstance(w, Sparse48MMA):
        if not (isinstance(x, NVFP4MMA) and isinstance(w, Sparse48MMA)):
            raise ValueError("tile images are taken for both operands or neither")
        M, N = x.rows, w.rows
        if x.cols != K or w.K != K:
            raise ValueError(f"K mismatch: {x.cols}, {w.K} vs {K}")
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=w.meta.device)
        xo = _Operand(NVFP4_B32_MMA, x.codes.data_ptr(), x.scales.data_ptr(), x.tensor_scale.data_ptr())
        wo = _SparseOperand(NVFP4_MMA, w.values.data_ptr(), w.scales.data_ptr(), w.tensor_scale.data_ptr(),
                            w.meta.data_ptr())
        _call("sp24_gemm_sparse48", ctypes.byref(xo), ctypes.byref(wo), M, N, K, _ptr(out), _stream(stream))
        return out
    M = x.codes.shape[0]
    if x.codes.shape[1] * 2 != K:
        raise ValueError(f"K mismatch: {x.codes.shape[1] * 2} vs {K}")
    v = w.values
    N = v.codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=w.meta.device)
    xo = _Operand(NVFP4_B32, x.codes.data_ptr(), x.scales.data_ptr(), x.tensor_scale.data_ptr())
    wo = _SparseOperand(NVFP4, v.codes.data_ptr(), v.scales.data_ptr(), v.tensor_scale.data_ptr(), w.meta.data_ptr())
    _call("sp24_gemm_sparse48", ctypes.byref(xo), ctypes.byref(wo), M, N, K, _ptr(out), _stream(stream))
    return out


def _sparse_operand(w: "Sparse24") -> _SparseOperand:
    v = w.values
    if isinstance(v, NVFP4Tensor):
        return _SparseOperand(NVFP4, v.codes.data_ptr(), v.scales.data_ptr(), v.tensor_scale.data_ptr(),
                              w.meta.data_ptr())
    _cuda(v, "values")
    return _SparseOperand(_dtype_code(v), v.data_ptr(), None, None, w.meta.data_ptr())


def _both_forms(x, w_dense, w_sparse: "Sparse24"):
    M, K = _rows_k(x)
    N, Kw = _rows_k(w_dense)
    if K != Kw:
        raise ValueError(f"K mismatch: {K} vs {Kw}")
    ws = max(gemm_workspace_bytes(x, w_dense, False, M, N, K), gemm_workspace_bytes(x, w_sparse, True, M, N, K))
    return M, N, K, ws


def gemm_choice(x_format: int, w_format: int, M: int, N: int, K: int) -> tuple:
    """(use_sparse, measured): the dense / 2:4 decision for a shape (host only)."""
    u, m = ctypes.c_int(0), ctypes.c_int(0)
    _call("sp24_gemm_choice", x_format, w_format, M, N, K, ctypes.byref(u), ctypes.byref(m))
    return bool(u.value), bool(m.value)


def gemm_choice_reset() -> None:
    _call("sp24_gemm_choice_reset")


def gemm_select(x, w_dense, w_sparse: "Sparse24", reps: int = 10, out=None, workspace=None, stream=None) -> dict:
    """Times the dense and the 2:4 GEMM of this shape, records the faster one (synchronises)."""
    M, N, K, ws_bytes = _both_forms(x, w_dense, w_sparse)
    dev = w_sparse.meta.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    xo, wd, wsp = _operand(x), _operand(w_dense), _sparse_operand(w_sparse)
    u, td, tsp = ctypes.c_int(0), ctypes.c_float(0), ctypes.c_float(0)
    _call("sp24_gemm_select", ctypes.byref(xo), ctypes.byref(wd), ctypes.byref(wsp), M, N, K, _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), reps, ctypes.byref(u),
          ctypes.byref(td), ctypes.byref(tsp), _stream(stream))
    return {"use_sparse": bool(u.value), "us_dense": td.value, "us_sparse": tsp.value}


def gemm_auto(x, w_dense, w_sparse: "Sparse24", out=None, workspace=None, stream=None):
    """Y[M, N] from whichever form sp24_gemm_choice names; returns (Y, used_sparse)."""
    M, N, K, ws_bytes = _both_forms(x, w_dense, w_sparse)
    dev = w_sparse.meta.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    xo, wd, wsp = _operand(x), _operand(w_dense), _sparse_operand(w_sparse)
    u = ctypes.c_int(0)
    _call("sp24_gemm_auto", ctypes.byref(xo), ctypes.byref(wd), ctypes.byref(wsp), M, N, K, _ptr(out),
          _ptr(workspace), 0 if workspace is None else workspace.numel(), ctypes.byref(u), _stream(stream))
    return out, bool(u.value)


def grouped_workspace_bytes(T: int, topk: int, E: int) -> int:
    n = ctypes.c_int64(0)
    _call("sp24_gemm_grouped_workspace_size", T, topk, E, ctypes.byref(n))
    return n.value


def gemm_grouped(x, routing: torch.Tensor, w, E: int, N: int, K: int, out=None, workspace=None,
                 stream=None) -> torch.Tensor:
    """Routed-expert GEMM: Y[t, s, :] = x[t] @ W[routing[t, s]]^T with the E experts stacked as
    one [E*N, K] operand (16-bit tensor, NVFP4Tensor, or Sparse24 of those).  An id of -1 is a slot
    without an expert: zeros."""
    _cuda(routing, "routing")
    T, topk = routing.shape
    dev = routing.device
    if out is None:
        out = torch.empty((T, topk, N), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(grouped_workspace_bytes(T, topk, E), dtype=torch.uint8, device=dev)
    xo = _operand(x)
    if isinstance(w, Sparse24):
        v = w.values
        if isinstance(v, NVFP4Tensor):
            so = _SparseOperand(NVFP4, v.codes.data_ptr(), v.scales.data_ptr(), v.tensor_scale.data_ptr(),
                                w.meta.data_ptr())
        else:
            so = _SparseOperand(_dtype_code(v), v.data_ptr(), None, None, w.meta.data_ptr())
        dense_p, sparse_p = None, ctypes.byref(so)
    else:
        do = _operand(w)
        dense_p, sparse_p = ctypes.byref(do), None
    _call("sp24_gemm_grouped", ctypes.byref(xo), _ptr(routing), T, topk, dense_p, sparse_p, E, N, K,
          _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    return out


def kernel_launches() -> int:
    """Kernels this library has launched in this process (host-side count)."""
    return int(lib().sp24_kernel_launches())


def last_device_error(stream=None) -> int:
    return int(lib().sp24_last_device_error(_stream(stream)))


def sizes(op: int, dtype: int, shape) -> dict:
    """Host-side size arithmetic of the compressed and NVFP4 forms (no device access)."""
    out = [ctypes.c_int64(0) for _ in range(5)]
    _call("sp24_sizes", op, dtype, _shape(shape), len(shape), *[ctypes.byref(o) for o in out])
    keys = ("groups", "values_bytes", "meta_bytes", "nvfp4_codes_bytes", "nvfp4_scales_bytes")
    return {k: o.value for k, o in zip(keys, out)}


def _interleave(a: torch.Tensor, b: torch.Tensor, rows: int, block_rows: int = 16, stream=None) -> torch.Tensor:
    _cuda(a, "a")
    _cuda(b, "b")
    if a.shape != b.shape or a.dtype != b.dtype:
        raise ValueError("interleave wants two tensors of one shape and dtype")
    row_bytes = a.numel() * a.element_size() // rows
    out = torch.empty((2 * rows, row_bytes), dtype=torch.uint8, device=a.device)
    _call("sp24_interleave_rows", _ptr(a), _ptr(b), rows, row_bytes, block_rows, _ptr(out), _stream(stream))
    return out


def pack_gate_up(gate, up, stream=None):
    """The expert block's gate / up operand: the stacked gate and up weights [E*F, H] (NVFP4Tensor,
    or Sparse24 of NVFP4Tensor values, sharing one tensor scale) packed in 16-row blocks."""
    if isinstance(gate, Sparse24):
        gv, uv = gate.values, up.values
        rows = gv.codes.shape[0]
        vals = NVFP4Tensor(_interleave(gv.codes, uv.codes, rows, stream=stream),
                           _interleave(gv.scales, uv.scales, rows, stream=stream), gv.tensor_scale.clone())
        return Sparse24(vals, _interleave(gate.meta, up.meta, rows, stream=stream).reshape(-1))
    rows = gate.codes.shape[0]
    return NVFP4Tensor(_interleave(gate.codes, up.codes, rows, stream=stream),
                       _interleave(gate.scales, up.scales, rows, stream=stream), gate.tensor_scale.clone())


def moe_block_workspace_bytes(T: int, topk: int, E: int, H: int, F: int) -> int:
    n = ctypes.c_int64(0)
    _call("sp24_moe_block_workspace_size", T, topk, E, H, F, ctypes.byref(n))
    return n.value


def moe_block(x: torch.Tensor, routing: torch.Tensor, router_w: torch.Tensor, w_gate_up, w_down, E: int, H: int,
              F: int, out=None, workspace=None, stream=None) -> torch.Tensor:
    """y[T, H] fp32 = sum_s r[t, s] * (SiLU(x Wg^T) * (x Wu^T)) Wd^T over the routed experts;
    w_gate_up from pack_gate_up, w_down [E*H, F]; each an NVFP4Tensor or a Sparse24 of one.  A slot
    with the id -1 adds nothing."""
    _cuda(routing, "routing")
    _cuda(router_w, "router_w")
    T, topk = routing.shape
    dev = routing.device
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(moe_block_workspace_bytes(T, topk, E, H, F), dtype=torch.uint8, device=dev)
    xo = _operand(x)
    gd = gs = dd = ds = None
    if isinstance(w_gate_up, Sparse24):
        gs = ctypes.byref(_sparse_operand(w_gate_up))
    else:
        gd = ctypes.byref(_operand(w_gate_up))
    if isinstance(w_down, Sparse24):
        ds = ctypes.byref(_sparse_operand(w_down))
    else:
        dd = ctypes.byref(_operand(w_down))
    _call("sp24_moe_block", ctypes.byref(xo), _ptr(routing), _ptr(router_w), T, topk, gd, gs, dd, ds, E, H, F,
          _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    return out


# ---------------------------------------------------------------------------- routed feed-forward

def _placed(impl):
    """Runs `impl` on the device of its first tensor and on `stream` (default: that device's current
    stream), with what it allocates belonging to that stream.  Arguments after `out` are by name."""
    name = next(iter(inspect.signature(impl).parameters))

    @functools.wraps(impl)
    def call(*args, stream=None, **kw):
        t = args[0] if args else kw.get(name)
        if type(t) is W4Tensor:
            t = t.codes
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
        if stream is None and t.get_device() == _current_device():
            return impl(*args, **kw)
        if stream is not None and stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.device(t.device), torch.cuda.stream(stream):
            return impl(*args, **kw)
    return call


# the current device, and a device's current stream as the runtime's own handle, without the
# initialisation check of torch.cuda's functions (a CUDA tensor is at hand)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _arg(t, name: str, dev: int, shape, *dtypes) -> int:
    """The address of an argument that has to be contiguous, on device `dev`, and of this shape and
    type."""
    try:
        if t.get_device() == dev and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(st: int, fn: str) -> None:
    if st != OK:
        raise SP24Error(st, fn)


_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_HALVES = (torch.bfloat16, torch.float16)


def _dims(t: torch.Tensor, name: str, n: int):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, not {t.dim()}")
    return t.shape


class MoeSorted(NamedTuple):
    """Tokens in the order of their experts (sp24_moe_sort) with the tables of that order."""
    xs: Optional[torch.Tensor]  # [T * topk, H] or None
    pos: torch.Tensor           # int32 [T, topk]: row of (token, slot), -1 for an empty slot
    src: torch.Tensor           # int32 [T * topk]: token * topk + slot of a row, -1 behind the last
    row_expert: torch.Tensor    # int32 [T * topk]: expert of a row, -1 behind the last
    offsets: torch.Tensor       # int32 [E + 1]


@_placed
def moe_route(logits: torch.Tensor, topk: int, scoring: int = ROUTE_SOFTMAX, renormalize: bool = True, out=None):
    """(routing int32 [T, topk], router_w fp32 [T, topk]) of router logits [T, E]: the topk largest
    logits (ties to the lower expert) and their softmax or sigmoid weights."""
    dev = logits.get_device()
    T, E = _dims(logits, "logits", 2)
    lp = _arg(logits, "logits", dev, logits.shape, *_FLOATS)
    if out is None:
        out = (torch.empty((T, topk), dtype=torch.int32, device=dev),
               torch.empty((T, topk), dtype=torch.float32, device=dev))
    routing, w = out
    _check((_lib or lib()).sp24_moe_route(lp, _DT[logits.dtype], T, E, topk, scoring, bool(renormalize),
                                _arg(routing, "routing", dev, (T, topk), torch.int32),
                                _arg(w, "router_w", dev, (T, topk), torch.float32), _raw_stream(dev)), "sp24_moe_route")
    return routing, w


@_placed
def moe_route_backward(d_router_w: torch.Tensor, logits: torch.Tensor, routing: torch.Tensor,
                       scoring: int = ROUTE_SOFTMAX, renormalize: bool = True, out=None) -> torch.Tensor:
    """The gradient of moe_route's logits (their type, [T, E]) from that of its weights."""
    dev = logits.get_device()
    T, E = _dims(logits, "logits", 2)
    topk = _dims(routing, "routing", 2)[1]
    lp = _arg(logits, "logits", dev, logits.shape, *_FLOATS)
    if out is None:
        out = torch.empty_like(logits)
    _check((_lib or lib()).sp24_moe_route_backward(lp, _DT[logits.dtype], _arg(routing, "routing", dev, (T, topk), torch.int32),
                                         _arg(d_router_w, "d_router_w", dev, (T, topk), torch.float32), T, E, topk,
                                         scoring, bool(renormalize), _arg(out, "out", dev, (T, E), logits.dtype),
                                         _raw_stream(dev)), "sp24_moe_route_backward")
    return out


@functools.lru_cache(maxsize=1024)
def moe_sort_workspace_bytes(T: int, topk: int, E: int) -> int:
    n = ctypes.c_int64(0)
    _call("sp24_moe_sort_workspace_size", T, topk, E, ctypes.byref(n))
    return n.value


def _sort(x, routing, E: int, out, workspace) -> MoeSorted:
    dev = routing.get_device()
    T, topk = _dims(routing, "routing", 2)
    n = T * topk
    xp = xsp = None
    H, dt = 0, F32
    if x is not None:
        H, dt = _dims(x, "x", 2)[1], _dtype_code(x)
        xp = _arg(x, "x", dev, (T, H), *_FLOATS)
    if out is None:
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
        out = (None if x is None else torch.empty((n, H), dtype=x.dtype, device=dev), i32(T, topk), i32(n), i32(n), i32(E + 1))
    xs, pos, src, row_expert, offsets = out
    if x is not None:
        xsp = _arg(xs, "xs", dev, (n, H), x.dtype)
    ws = moe_sort_workspace_bytes(T, topk, E)
    if workspace is None and ws:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    wp, wn = (None, 0) if workspace is None else (_arg(workspace, "workspace", dev, workspace.shape, torch.uint8), workspace.numel())
    _check((_lib or lib()).sp24_moe_sort(xp, dt, _arg(routing, "routing", dev, (T, topk), torch.int32), T, topk, E, H, xsp,
                               _arg(pos, "pos", dev, (T, topk), torch.int32), _arg(src, "src", dev, (n,), torch.int32),
                               _arg(row_expert, "row_expert", dev, (n,), torch.int32),
                               _arg(offsets, "offsets", dev, (E + 1,), torch.int32), wp, wn, _raw_stream(dev)),
           "sp24_moe_sort")
    return MoeSorted(xs, pos, src, row_expert, offsets)


@_placed
def moe_sort(x: torch.Tensor, routing: torch.Tensor, E: int, out=None, workspace=None) -> MoeSorted:
    """x [T, H] in the order of the experts in routing [T, topk] (stable), with the tables of that
    order.  An id of -1 is an empty slot; rows of xs behind the last expert's are not written (when
    allocated here they hold anything)."""
    return _sort(x, routing, E, out, workspace)


@_placed
def moe_sort_tables(routing: torch.Tensor, E: int, out=None, workspace=None) -> MoeSorted:
    """moe_sort without the rows: the tables only (xs is None)."""
    return _sort(None, routing, E, out, workspace)


def _unsort(ys, pos, router_w, dtype, out):
    dev = ys.get_device()
    rows, H = _dims(ys, "ys", 2)
    T, topk = _dims(pos, "pos", 2)
    yp = _arg(ys, "ys", dev, ys.shape, *_FLOATS)
    if out is None:
        out = torch.empty((T, H), dtype=dtype or ys.dtype, device=dev)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, not {out.dtype}")
    wp = None if router_w is None else _arg(router_w, "router_w", dev, (T, topk), torch.float32)
    _check((_lib or lib()).sp24_moe_unsort(yp, _DT[ys.dtype], _arg(pos, "pos", dev, (T, topk), torch.int32), wp, T, topk, rows, H,
                                 _arg(out, "out", dev, (T, H), *_FLOATS), _DT[out.dtype], _raw_stream(dev)),
           "sp24_moe_unsort")
    return out


@_placed
def moe_sort_backward(dxs: torch.Tensor, pos: torch.Tensor, out=None) -> torch.Tensor:
    """The gradient of moe_sort's x from that of xs: each token's rows summed (fp32, slot order)."""
    return _unsort(dxs, pos, None, dxs.dtype, out)


@_placed
def moe_unsort(ys: torch.Tensor, pos: torch.Tensor, router_w: Optional[torch.Tensor] = None, dtype=None,
               out=None) -> torch.Tensor:
    """y[t] = sum_s router_w[t, s] ys[pos[t, s]] (None: weights of 1), in ys's type or `dtype`."""
    return _unsort(ys, pos, router_w, dtype, out)


@_placed
def moe_unsort_backward(dy: torch.Tensor, ys: torch.Tensor, pos: torch.Tensor, router_w: Optional[torch.Tensor] = None,
                        out=None):
    """(dys, d_router_w) of moe_unsort; rows of dys that no slot names are not written (zeros when
    allocated here, which takes a fill of the whole of dys first: pass `out` where every row is named
    or the others do not count).  Without router_w, d_router_w is None."""
    dev = ys.get_device()
    rows, H = _dims(ys, "ys", 2)
    T, topk = _dims(pos, "pos", 2)
    yp = _arg(ys, "ys", dev, ys.shape, *_FLOATS)
    if out is None:
        out = (torch.zeros_like(ys), None if router_w is None else torch.empty((T, topk), dtype=torch.float32, device=dev))
    dys, dw = out
    wp = None if router_w is None else _arg(router_w, "router_w", dev, (T, topk), torch.float32)
    dwp = None if dw is None else _arg(dw, "d_router_w", dev, (T, topk), torch.float32)
    _check((_lib or lib()).sp24_moe_unsort_backward(_arg(dy, "dy", dev, (T, H), *_FLOATS), _DT[dy.dtype], yp, _DT[ys.dtype],
                                          _arg(pos, "pos", dev, (T, topk), torch.int32), wp, T, topk, rows, H,
                                          _arg(dys, "dys", dev, (rows, H), ys.dtype), dwp, _raw_stream(dev)),
           "sp24_moe_unsort_backward")
    return dys, dw


# ---------------------------------------------------------------------------- 4-bit group weights

class W4Tensor(NamedTuple):
    """4-bit weights with group scales: codes uint8 [rows, K/2] (entry 2i in the low nibble), scales
    [rows, K/group] f16 / bf16, zeros uint8 [rows, K/group] or None (8): value = (q - z) * s."""
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor] = None


_pack_w4 = struct.Struct("iiPPP").pack  # _W4Operand's bytes, cheaper to make


def _w4(w: W4Tensor, dev: int):
    """(C operand, rows, K) of 4-bit weights on `dev`."""
    rows, half = _dims(w.codes, "codes", 2)
    K = 2 * half
    groups = _dims(w.scales, "scales", 2)[1]
    group = K // groups if groups else 128
    if groups * group != K:
        raise ValueError(f"{groups} groups do not divide {K} entries")
    op = _pack_w4(_DT.get(w.scales.dtype, -1), group, _arg(w.codes, "codes", dev, (rows, half), torch.uint8),
                  _arg(w.scales, "scales", dev, (rows, groups), *_HALVES),
                  0 if w.zeros is None else _arg(w.zeros, "zeros", dev, (rows, groups), torch.uint8))
    return op, rows, K


@_placed
def quantize_w4(w: torch.Tensor, group: int = 128, zeros: bool = False, out: Optional[W4Tensor] = None) -> W4Tensor:
    """4-bit codes of a 16-bit weight [rows, K], rounded to nearest, with one scale per `group`
    entries (symmetric), or with a zero point beside each scale."""
    dev = w.get_device()
    R, K = _dims(w, "w", 2)
    wp = _arg(w, "w", dev, w.shape, *_HALVES)
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"groups of 32, 64 or 128 that divide K = {K}, not {group}")
    if out is None:
        out = W4Tensor(torch.empty((R, K // 2), dtype=torch.uint8, device=dev),
                       torch.empty((R, K // group), dtype=w.dtype, device=dev),
                       torch.empty((R, K // group), dtype=torch.uint8, device=dev) if zeros else None)
    elif (out.zeros is not None) != bool(zeros):
        raise ValueError("out.zeros must be there exactly where zeros is asked for")
    zp = _arg(out.zeros, "zeros", dev, (R, K // group), torch.uint8) if zeros else None
    _check((_lib or lib()).sp24_quantize_w4(wp, _DT[w.dtype], R, K, group, bool(zeros),
                                  _arg(out.codes, "codes", dev, (R, K // 2), torch.uint8),
                                  _arg(out.scales, "scales", dev, (R, K // group), w.dtype), zp, _raw_stream(dev)),
           "sp24_quantize_w4")
    return out


@_placed
def dequantize_w4(w: W4Tensor, dtype=torch.float32, out=None) -> torch.Tensor:
    """The values (q - z) * s of 4-bit weights, rounded once to `dtype`."""
    dev = w.codes.get_device()
    op, rows, K = _w4(w, dev)
    if dtype not in _FLOATS:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, not {dtype}")
    if out is None:
        out = torch.empty((rows, K), dtype=dtype, device=dev)
    _check((_lib or lib()).sp24_dequantize_w4(op, rows, K, _DT[dtype], _arg(out, "out", dev, (rows, K), dtype),
                                    _raw_stream(dev)), "sp24_dequantize_w4")
    return out


def _gemv_out(x, rows: int, N: int, act: int, dtype, out):
    cols = N // 2 if act == ACT_SWIGLU else N
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype or (x.dtype if act == ACT_SWIGLU else torch.float32), device=x.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, not {out.dtype}")
    return out, _arg(out, "out", x.get_device(), (rows, cols), torch.float32, x.dtype)


@_placed
def gemv_w4(x: torch.Tensor, w: W4Tensor, act: int = ACT_NONE, dtype=None, out=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ value(w)[N, K]^T for a few rows x (f16 / bf16), fp32 (or x's type by
    `dtype`); ACT_SWIGLU: w holds gate rows then up rows, y[M, N/2] = SiLU(gate) * up in x's type.
    For many rows: gemm_dense(x, dequantize_w4(w, x.dtype))."""
    dev = x.get_device()
    M, K = _dims(x, "x", 2)
    xp = _arg(x, "x", dev, x.shape, *_HALVES)
    op, N, Kw = _w4(w, dev)
    if K != Kw:
        raise ValueError(f"K mismatch: {K} vs {Kw}")
    out, yp = _gemv_out(x, M, N, act, dtype, out)
    _check((_lib or lib()).sp24_gemv_w4(xp, _DT[x.dtype], op, M, N, K, act, yp, _DT[out.dtype], _raw_stream(dev)),
           "sp24_gemv_w4")
    return out


@_placed
def gemv_w4_grouped(xs: torch.Tensor, w: W4Tensor, offsets: torch.Tensor, act: int = ACT_NONE, dtype=None,
                    out=None) -> torch.Tensor:
    """gemv_w4 over rows in expert order (moe_sort's xs and offsets [E + 1]) with the E matrices
    stacked in w; rows from offsets[E] on are not written (zeros when allocated here, which takes a
    fill first: pass `out` to save it).  For many rows: gemm_grouped(xs, row_expert[:, None],
    dequantize_w4(w, xs.dtype), E, N, K)."""
    dev = xs.get_device()
    R, K = _dims(xs, "xs", 2)
    xp = _arg(xs, "xs", dev, xs.shape, *_HALVES)
    op, rows, Kw = _w4(w, dev)
    E = _dims(offsets, "offsets", 1)[0] - 1
    if K != Kw:
        raise ValueError(f"K mismatch: {K} vs {Kw}")
    if E < 1 or rows % E:
        raise ValueError(f"{rows} weight rows are not those of {E} experts")
    N = rows // E
    if out is None:
        cols = N // 2 if act == ACT_SWIGLU else N
        out = torch.zeros((R, cols), dtype=dtype or (xs.dtype if act == ACT_SWIGLU else torch.float32), device=dev)
    out, yp = _gemv_out(xs, R, N, act, dtype, out)
    _check((_lib or lib()).sp24_gemv_w4_grouped(xp, _DT[xs.dtype], op, _arg(offsets, "offsets", dev, (E + 1,), torch.int32),
                                      R, E, N, K, act, yp, _DT[out.dtype], _raw_stream(dev)), "sp24_gemv_w4_grouped")
    return out
