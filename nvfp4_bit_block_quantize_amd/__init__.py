"""Python binding of libnvfp4.so (NVFP4 quantize / RHT-quantize / dequantize / GEMM on MI355X).

Argument marshalling only: PyTorch provides device memory and the current HIP stream, every step
of the computation runs in the library's HIP kernels.  The functions carry the C ABI's names
(include/nvfp4.h).  If the shared library has not been built the import of any function raises;
there is no fallback path.

    import torch, nvfp4_bit_block_quantize_amd as nv
    qx = nv.nvfp4_quantize(x)                                   # 1D blocks, nearest-even
    qw = nv.nvfp4_quantize(w, flags=nv.NVFP4_BLOCK2D)           # 16x16 weight tiles
    y  = nv.nvfp4_gemm(qx, qw, out_dtype=torch.bfloat16)        # y = x_hat @ w_hat^T
"""
from __future__ import annotations

import array
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

__all__ = [
    "NVFP4_OK", "NVFP4_ERR_NULL", "NVFP4_ERR_SHAPE", "NVFP4_ERR_ALIGN", "NVFP4_ERR_UNSUPPORTED",
    "NVFP4_ERR_HIP", "NVFP4_F32", "NVFP4_BF16", "NVFP4_COLWISE", "NVFP4_BLOCK2D", "NVFP4_SR",
    "NVFP4_FOUR_OVER_SIX", "NVFP4_TS_FOR_FOUR", "NVFP4_SCALE_SEARCH", "NVFP4Error", "NVFP4Tensor", "library_path", "lib",
    "nvfp4_workspace_size", "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_rht_quantize", "nvfp4_dequantize",
    "nvfp4_gemm", "nvfp4_gemm_nvfp4_out", "nvfp4_scale_from_amax", "nvfp4_gemm_w4a16", "nvfp4_transpose", "nvfp4_status_string", "empty_like_quantized",
    "NVFP4_ROUTE_SIGMOID", "NVFP4_ROUTE_RENORM", "NVFP4_ROUTE_GROUP_SUM2", "NVFP4_NORM_ONE_PLUS", "MoEPlan", "Int8Tensor",
    "BlockNorm", "BlockNormGrads", "nvfp4_moe_route", "nvfp4_moe_route_backward", "nvfp4_moe_plan", "nvfp4_moe_gather",
    "nvfp4_moe_combine", "nvfp4_moe_combine_backward", "nvfp4_int8_quantize", "nvfp4_int8_gemm", "nvfp4_block_norm",
    "nvfp4_block_norm_backward", "NVFP4_GRAD_MAX", "MoEBalance", "nvfp4_moe_balance", "nvfp4_moe_balance_backward",
    "nvfp4_grad_norm", "nvfp4_grad_clip", "NVFP4_ADAPTER_GATHER", "NVFP4_ADAPTER_BY_TOKEN", "Adapters", "AdapterGrads",
    "nvfp4_adapter", "nvfp4_adapter_backward",
]

NVFP4_OK, NVFP4_ERR_NULL, NVFP4_ERR_SHAPE, NVFP4_ERR_ALIGN, NVFP4_ERR_UNSUPPORTED, NVFP4_ERR_HIP = range(6)
NVFP4_F32, NVFP4_BF16 = 0, 1
NVFP4_COLWISE, NVFP4_BLOCK2D, NVFP4_SR, NVFP4_FOUR_OVER_SIX = 1, 2, 4, 8
NVFP4_TS_FOR_FOUR, NVFP4_SCALE_SEARCH = 16, 32
NVFP4_ROUTE_SIGMOID, NVFP4_ROUTE_RENORM, NVFP4_ROUTE_GROUP_SUM2 = 1, 2, 4
NVFP4_NORM_ONE_PLUS, NVFP4_NORM_TOKEN_GATE = 1, 2
NVFP4_GRAD_MAX = 1
NVFP4_ADAPTER_GATHER, NVFP4_ADAPTER_BY_TOKEN = 1, 2

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


def library_path() -> str:
    return os.path.join(_HERE, "libnvfp4.so")


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("k", ctypes.c_int64), ("flags", ctypes.c_uint32)]


def lib():
    """The loaded libnvfp4.so.  Raises if it has not been built (python -m
    nvfp4_bit_block_quantize_amd.build)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libnvfp4.so not built at {path}; run python -m nvfp4_bit_block_quantize_amd.build")
        L = ctypes.CDLL(path)
        P, i64, u32, u64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int32
        TP = ctypes.POINTER(_Tensor)
        L.nvfp4_workspace_size.argtypes = [i64, i64, u32]
        L.nvfp4_workspace_size.restype = ctypes.c_size_t
        L.nvfp4_quantize.argtypes = [P, ctypes.c_int, i64, i64, i64, u32, u64, u32, TP, P, P]
        L.nvfp4_quantize.restype = ctypes.c_int
        L.nvfp4_quantize_noalloc.argtypes = [P, ctypes.c_int, i64, i64, i64, u32, u64, u32, TP, P]
        L.nvfp4_quantize_noalloc.restype = ctypes.c_int
        L.nvfp4_rht_quantize.argtypes = [P, ctypes.c_int, i64, i64, i64, u32, u64, u32, u64, P, TP, P, P]
        L.nvfp4_rht_quantize.restype = ctypes.c_int
        L.nvfp4_quantize_grouped.argtypes = [P, ctypes.c_int, i64, i64, i64, i64, i64, u32, u64, u32, TP, P, P]
        L.nvfp4_quantize_grouped.restype = ctypes.c_int
        L.nvfp4_dequantize.argtypes = [TP, P, ctypes.c_int, i64, P]
        L.nvfp4_dequantize.restype = ctypes.c_int
        L.nvfp4_gemm.argtypes = [TP, TP, P, ctypes.c_int, i64, i32, ctypes.POINTER(ctypes.c_int64), P]
        L.nvfp4_gemm.restype = ctypes.c_int
        L.nvfp4_gemm_nvfp4_out.argtypes = [TP, TP, TP, P, i32, ctypes.POINTER(ctypes.c_int64), P]
        L.nvfp4_gemm_nvfp4_out.restype = ctypes.c_int
        L.nvfp4_scale_from_amax.argtypes = [P, P, P]
        L.nvfp4_scale_from_amax.restype = ctypes.c_int
        L.nvfp4_gemm_w4a16.argtypes = [P, ctypes.c_int, i64, i64, TP, P, ctypes.c_int, i64, P]
        L.nvfp4_gemm_w4a16.restype = ctypes.c_int
        L.nvfp4_transpose.argtypes = [TP, TP, P]
        L.nvfp4_transpose.restype = ctypes.c_int
        i, f32, size = ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        for name, res, args in (
                ("nvfp4_moe_workspace_size", size, [i64, i64, i32]),
                ("nvfp4_moe_route", i, [P, i, i64, i64, i64, P, i32, i32, i32, u32, f32, P, P, P, P, P, P, P]),
                ("nvfp4_moe_route_backward", i, [P, i, i64, i64, i64, P, P, i32, u32, f32, P, i64, P]),
                ("nvfp4_moe_plan", i, [P, i64, i32, i64, P, P, P, P, P]),
                ("nvfp4_moe_gather", i, [P, i, i64, i64, i64, P, i32, P, i64, P]),
                ("nvfp4_moe_combine", i, [P, i, i64, i64, i64, P, P, i32, P, i64, P]),
                ("nvfp4_moe_combine_backward", i, [P, i64, P, i64, i, i64, i64, P, P, P, i32, P, i64, P, P]),
                ("nvfp4_int8_quantize", i, [P, i, i64, i64, i64, P, P, P]),
                ("nvfp4_int8_gemm_workspace_size", size, [i64, i64, i64]),
                ("nvfp4_int8_gemm", i, [P, P, i64, P, P, i64, i64, i64, P, i, i64, i32, P, P, i32, P, P]),
                ("nvfp4_block_norm", i, [P, i, P, i, i64, i64, P, P, P, f32, f32, u32, P, P, P, P, P]),
                ("nvfp4_block_norm_workspace_size", size, [i64, i64]),
                ("nvfp4_block_norm_backward", i,
                 [P, P, P, i, P, i, i64, i64, P, P, P, f32, u32, P, P, P, P, P, P, P, P, P]),
                ("nvfp4_moe_balance_workspace_size", size, [i64, i64, i64]),
                ("nvfp4_moe_balance", i, [P, i, i64, i64, i64, P, i32, i64, u32, f32, P, P, P, P, P, P]),
                ("nvfp4_moe_balance_backward", i,
                 [P, i, i64, i64, i64, P, i32, i64, u32, f32, P, P, P, P, i64, P, i64, P]),
                ("nvfp4_adapter_workspace_size", size, [i64, i64, i64, i32, i32]),
                ("nvfp4_adapter_backward_workspace_size", size, [i64, i64, i64, i32, i32]),
                ("nvfp4_adapter", i, [P, i, i64, i64, P, P, P, i64, i64, i64, i32, i32, P, P, P, i32, u32, P, i64, P, i, i64, P, P, P]),
                ("nvfp4_adapter_backward", i,
                 [P, i, i64, P, i, i64, P, P, P, i64, i64, i64, i32, i32, P, P, P, u32, P, P, i64, P, i, i64, P, P, P, P]),
                ("nvfp4_grad_workspace_size", size, [i64, i64]),
                ("nvfp4_grad_norm", i, [P, P, P, i64, u32, P, P, P]),
                ("nvfp4_grad_clip", i, [P, P, P, P, i64, P, f32, f32, P])):
            getattr(L, name).argtypes, getattr(L, name).restype = args, res
        L.nvfp4_status_string.argtypes = [ctypes.c_int]
        L.nvfp4_status_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {nvfp4_status_string(status)}")
        self.status = status


def nvfp4_status_string(status: int) -> str:
    return lib().nvfp4_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


@dataclass
class NVFP4Tensor:
    """An NVFP4 tensor (logical [rows x k], k contiguous).  For a grouped GEMM weight the three
    buffers hold `groups` consecutive tensors of `rows` rows each."""
    data: torch.Tensor          # uint8 [groups*rows, k/2]
    scales: torch.Tensor        # uint8 [groups*rows, k/16] or [groups*rows/16, k/16]
    tensor_scale: torch.Tensor  # float32 [groups]
    rows: int
    k: int
    flags: int = 0
    groups: int = 1

    def descriptor(self) -> _Tensor:
        return _Tensor(self.data.data_ptr() if self.data.numel() else None,
                       self.scales.data_ptr() if self.scales.numel() else None,
                       self.tensor_scale.data_ptr(), self.rows, self.k, self.flags & NVFP4_BLOCK2D)

    @property
    def block2d(self) -> bool:
        return bool(self.flags & NVFP4_BLOCK2D)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return NVFP4_F32
    if t == torch.bfloat16:
        return NVFP4_BF16
    raise TypeError(f"unsupported dtype {t}; NVFP4 inputs are float32 or bfloat16")


def _stream_handle(device: torch.device):
    if device.type != "cuda":
        return None
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None or t.numel() == 0 else ctypes.c_void_p(t.data_ptr())


def nvfp4_workspace_size(rows: int, cols: int, flags: int = 0) -> int:
    return int(lib().nvfp4_workspace_size(rows, cols, flags))


def empty_like_quantized(rows: int, k: int, flags: int, device, groups: int = 1) -> NVFP4Tensor:
    """Allocate the output buffers of an NVFP4 tensor of logical shape [rows x k]."""
    data = torch.empty((groups * rows, k // 2), dtype=torch.uint8, device=device)
    if flags & NVFP4_BLOCK2D:
        scales = torch.empty((groups * rows // 16, k // 16), dtype=torch.uint8, device=device)
    else:
        scales = torch.empty((groups * rows, k // 16), dtype=torch.uint8, device=device)
    ts = torch.empty((groups,), dtype=torch.float32, device=device)
    return NVFP4Tensor(data, scales, ts, rows, k, flags & NVFP4_BLOCK2D, groups)


def _logical(x: torch.Tensor, flags: int):
    if x.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = x.shape
    return (cols, rows) if flags & NVFP4_COLWISE else (rows, cols)


def _ld(x: torch.Tensor) -> int:
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be row-major with unit column stride")
    return max(int(x.stride(0)), int(x.shape[1]), 1)


def nvfp4_quantize(x: torch.Tensor, flags: int = 0, seed: int = 0, stream_id: int = 0,
                   out: Optional[NVFP4Tensor] = None, workspace: Optional[torch.Tensor] = None) -> NVFP4Tensor:
    """Quantize x (float32 / bfloat16 [rows x cols]) to NVFP4 (see include/nvfp4.h)."""
    R, K = _logical(x, flags)
    if out is None:
        out = empty_like_quantized(R, K, flags, x.device)
    if workspace is None:
        workspace = torch.empty(nvfp4_workspace_size(*x.shape, flags) // 4, dtype=torch.int32, device=x.device)
    desc = out.descriptor()
    st = lib().nvfp4_quantize(_ptr(x), _dtype_code(x.dtype), x.shape[0], x.shape[1], _ld(x), flags, seed & (2**64 - 1),
                              stream_id, ctypes.byref(desc), _ptr(workspace), _stream_handle(x.device))
    _check(st, "nvfp4_quantize")
    return out


def nvfp4_quantize_noalloc(x: torch.Tensor, out: NVFP4Tensor, flags: int = 0, seed: int = 0,
                           stream_id: int = 0) -> NVFP4Tensor:
    """nvfp4_quantize into caller-allocated `out`, with the amax workspace in the library's own
    device array: the call allocates nothing (see include/nvfp4.h)."""
    desc = out.descriptor()
    st = lib().nvfp4_quantize_noalloc(_ptr(x), _dtype_code(x.dtype), x.shape[0], x.shape[1], _ld(x), flags,
                                      seed & (2**64 - 1), stream_id, ctypes.byref(desc), _stream_handle(x.device))
    _check(st, "nvfp4_quantize_noalloc")
    return out


def nvfp4_quantize_grouped(x: torch.Tensor, flags: int = 0, seed: int = 0, stream_id: int = 0,
                           out: Optional[NVFP4Tensor] = None, workspace: Optional[torch.Tensor] = None) -> NVFP4Tensor:
    """Quantize each x[g] of x (float32 / bfloat16 [groups x rows x cols], each x[g] with unit column
    stride) with its own tensor scale, group g with stream id stream_id + g, into one group-contiguous
    NVFP4 tensor (the grouped GEMM's weight layout; see include/nvfp4.h)."""
    if x.dim() != 3:
        raise ValueError("x must be [groups, rows, cols]")
    G, rows, cols = x.shape
    if G < 1:
        raise ValueError("x needs at least one group")
    R, K = _logical(x[0], flags)
    if out is None:
        out = empty_like_quantized(R, K, flags, x.device, groups=G)
    if workspace is None:
        workspace = torch.empty(G * nvfp4_workspace_size(rows, cols, flags) // 4, dtype=torch.int32, device=x.device)
    desc = out.descriptor()
    ldx = _ld(x[0])
    st = lib().nvfp4_quantize_grouped(_ptr(x), _dtype_code(x.dtype), G, rows, cols, ldx, x.stride(0) if G > 1 else 0,
                                      flags, seed & (2**64 - 1), stream_id, ctypes.byref(desc), _ptr(workspace),
                                      _stream_handle(x.device))
    _check(st, "nvfp4_quantize_grouped")
    return out


def nvfp4_rht_quantize(x: torch.Tensor, sign_seed: int, flags: int = 0, seed: int = 0, stream_id: int = 0,
                       rht_out: Optional[torch.Tensor] = None, out: Optional[NVFP4Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> NVFP4Tensor:
    """16x16 random Hadamard transform along K, then quantize (see include/nvfp4.h).  If rht_out
    (float32 [R x K]) is given, the transformed matrix is written to it as well."""
    R, K = _logical(x, flags)
    if out is None:
        out = empty_like_quantized(R, K, flags, x.device)
    if workspace is None:
        workspace = torch.empty(nvfp4_workspace_size(*x.shape, flags) // 4, dtype=torch.int32, device=x.device)
    desc = out.descriptor()
    st = lib().nvfp4_rht_quantize(_ptr(x), _dtype_code(x.dtype), x.shape[0], x.shape[1], _ld(x), flags,
                                  seed & (2**64 - 1), stream_id, sign_seed & (2**64 - 1), _ptr(rht_out),
                                  ctypes.byref(desc), _ptr(workspace), _stream_handle(x.device))
    _check(st, "nvfp4_rht_quantize")
    return out


def nvfp4_dequantize(t: NVFP4Tensor, dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    if out is None:
        out = torch.empty((t.rows, t.k), dtype=dtype, device=t.data.device)
    desc = t.descriptor()
    st = lib().nvfp4_dequantize(ctypes.byref(desc), _ptr(out), _dtype_code(out.dtype), _ld(out),
                                _stream_handle(out.device))
    _check(st, "nvfp4_dequantize")
    return out


def nvfp4_gemm(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype: torch.dtype = torch.bfloat16,
               group_offsets: Optional[Sequence[int]] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = A_hat @ B_hat^T with FP32 accumulation.  Grouped: group_offsets (host ints, G+1) split
    A's rows; b holds G weights of b.rows rows each."""
    M, N = a.rows, b.rows
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.data.device)
    da, db = a.descriptor(), b.descriptor()
    if group_offsets is not None:
        offs = (ctypes.c_int64 * len(group_offsets))(*[int(v) for v in group_offsets])
        G = len(group_offsets) - 1
    else:
        offs, G = None, 1
    st = lib().nvfp4_gemm(ctypes.byref(da), ctypes.byref(db), _ptr(out), _dtype_code(out.dtype), _ld(out), G, offs,
                          _stream_handle(out.device))
    _check(st, "nvfp4_gemm")
    return out


def nvfp4_gemm_nvfp4_out(a: NVFP4Tensor, b: NVFP4Tensor, out: NVFP4Tensor, amax: Optional[torch.Tensor] = None,
                         group_offsets: Optional[Sequence[int]] = None) -> NVFP4Tensor:
    """out = Q(A_hat @ B_hat^T), quantized row-wise (1D, nearest-even) in the GEMM's epilogue with the
    tensor scale already in out.tensor_scale; if amax (float32 [1], device) is given, max |C| is
    folded into it (see include/nvfp4.h)."""
    da, db, dout = a.descriptor(), b.descriptor(), out.descriptor()
    if group_offsets is not None:
        offs = (ctypes.c_int64 * len(group_offsets))(*[int(v) for v in group_offsets])
        G = len(group_offsets) - 1
    else:
        offs, G = None, 1
    st = lib().nvfp4_gemm_nvfp4_out(ctypes.byref(da), ctypes.byref(db), ctypes.byref(dout), _ptr(amax), G, offs,
                                    _stream_handle(out.data.device))
    _check(st, "nvfp4_gemm_nvfp4_out")
    return out


def nvfp4_scale_from_amax(amax: torch.Tensor, ts: torch.Tensor) -> torch.Tensor:
    """ts = amax / 2688 on the device (both float32 [1])."""
    st = lib().nvfp4_scale_from_amax(_ptr(amax), _ptr(ts), _stream_handle(ts.device))
    _check(st, "nvfp4_scale_from_amax")
    return ts


def nvfp4_gemm_w4a16(a: torch.Tensor, b: NVFP4Tensor, out_dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = A @ B_hat^T with A a bf16 [M x K] device matrix (unit stride along K) and B an NVFP4
    weight [N x K]; FP32 accumulation (see include/nvfp4.h)."""
    if a.dim() != 2 or a.stride(1) != 1:
        raise ValueError("nvfp4_gemm_w4a16: A must be 2-D with unit stride along K")
    if a.dtype != torch.bfloat16:
        raise TypeError("nvfp4_gemm_w4a16: A must be bfloat16")
    M, N = a.shape[0], b.rows
    if a.shape[1] != b.k:
        raise ValueError(f"nvfp4_gemm_w4a16: A has K={a.shape[1]}, B has K={b.k}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    db = b.descriptor()
    st = lib().nvfp4_gemm_w4a16(_ptr(a), NVFP4_BF16, M, _ld(a), ctypes.byref(db), _ptr(out),
                                _dtype_code(out.dtype), _ld(out), _stream_handle(out.device))
    _check(st, "nvfp4_gemm_w4a16")
    return out


def nvfp4_transpose(t: NVFP4Tensor, out: Optional[NVFP4Tensor] = None) -> NVFP4Tensor:
    """Transpose of a 16x16-block-scaled NVFP4 tensor (see include/nvfp4.h): codes, scale grid and
    tensor scale of t^T, equal to quantizing the transposed matrix directly."""
    if out is None:
        out = empty_like_quantized(t.k, t.rows, NVFP4_BLOCK2D, t.data.device)
    din, dout = t.descriptor(), out.descriptor()
    st = lib().nvfp4_transpose(ctypes.byref(din), ctypes.byref(dout), _stream_handle(t.data.device))
    _check(st, "nvfp4_transpose")
    return out


# ---- the block around the quantized products ----------------------------------------------------------
@dataclass
class MoEPlan:
    """The order of a grouped product's rows (see nvfp4_moe_plan): slot t * top_k + j is token t's choice j."""
    offsets: torch.Tensor  # int32 [experts + 1], first row of each expert
    rows: torch.Tensor     # int32 [tokens * top_k], the slot of each row (-1: none)
    pos: torch.Tensor      # int32 [tokens, top_k], the row of each slot (-1: none)

    @property
    def experts(self) -> int:
        return self.offsets.shape[0] - 1

    @property
    def top_k(self) -> int:
        return self.pos.shape[1]


@dataclass
class Int8Tensor:
    """8-bit integers with one scale a row (logical [rows x k], k contiguous); a grouped product's weight
    holds `groups` consecutive tensors of `rows` rows each."""
    data: torch.Tensor    # int8 [groups*rows, k]
    scales: torch.Tensor  # float32 [groups*rows]
    rows: int
    k: int
    groups: int = 1


@dataclass
class BlockNorm:
    """What nvfp4_block_norm gives."""
    x: torch.Tensor            # the residual stream after the block
    n: Optional[torch.Tensor]  # its norm, the next block's input
    rstd: torch.Tensor         # float32 [2, tokens]: of the block's output and of x, where they are normed
    has_post: bool

    @property
    def rstd_post(self) -> Optional[torch.Tensor]:
        """float32 [tokens], for the backward call."""
        return self.rstd[0] if self.has_post else None

    @property
    def rstd_pre(self) -> Optional[torch.Tensor]:
        return self.rstd[1] if self.n is not None else None


@dataclass
class BlockNormGrads:
    """What nvfp4_block_norm_backward gives (None where the forward call had no such input)."""
    dx: torch.Tensor
    dy: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]


def _raw_stream(t: torch.Tensor):
    """The current stream of t's device, as a number (torch.cuda.current_stream builds an object first).  A tensor in
    host memory is refused: the kernels would read its address on the GPU."""
    if not t.is_cuda:
        raise NVFP4Error(NVFP4_ERR_UNSUPPORTED, f"tensors on {t.device}")
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _want(where: str, name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape, like: torch.Tensor):
    """A contiguous tensor of this dtype and shape on the device of `like`."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == like.device):
        return
    if t.dtype is not dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, is {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous {list(shape)}, is {list(t.shape)}")
    raise ValueError(f"{where}: {name} is on {t.device}, not {like.device}")


def _matrix(where: str, name: str, t: torch.Tensor) -> int:
    """Leading dimension of a matrix with unit column stride."""
    if t.dim() == 2:
        rows, cols = t.shape
        ld, unit = t.stride()
        if unit == 1 or cols <= 1:
            if rows <= 1:
                return cols
            if ld >= cols:
                return ld
            raise ValueError(f"{where}: rows of {name} overlap")
    raise ValueError(f"{where}: {name} must be 2-D with unit column stride")


def _empty_plan(tokens: int, top_k: int, experts: int, device) -> MoEPlan:
    i32 = torch.int32
    return MoEPlan(torch.empty(experts + 1, dtype=i32, device=device), torch.empty(tokens * top_k, dtype=i32, device=device),
                   torch.empty((tokens, top_k), dtype=i32, device=device))


def _scratch(where: str, workspace: Optional[torch.Tensor], size: int, like: torch.Tensor) -> Optional[torch.Tensor]:
    """The caller's workspace if it has `size` bytes on the device of `like`; one of that size if there is none."""
    if workspace is None:
        return torch.empty(size // 4, dtype=torch.int32, device=like.device) if size else None
    if size and (workspace.numel() * workspace.element_size() < size or not workspace.is_contiguous()
                 or workspace.device != like.device):
        raise ValueError(f"{where}: workspace must be contiguous and have {size} bytes on {like.device}, has "
                         f"{workspace.numel() * workspace.element_size()} on {workspace.device}")
    return workspace


def nvfp4_moe_route(logits: torch.Tensor, top_k: int, flags: int = 0, bias: Optional[torch.Tensor] = None,
                    num_groups: int = 1, group_top_k: int = 1, scale: float = 1.0, with_plan: bool = True,
                    workspace: Optional[torch.Tensor] = None):
    """Route tokens to experts from logits [tokens, experts] (float32 / bfloat16, unit column stride);
    returns (ids int32 [tokens, top_k], weights float32 [tokens, top_k], MoEPlan or None).  See
    include/nvfp4.h for the scores, groups, ties and closed experts."""
    ld = _matrix("nvfp4_moe_route", "logits", logits)
    T, E = logits.shape
    _want("nvfp4_moe_route", "bias", bias, torch.float32, (E,), logits)
    dev = logits.device
    ids = torch.empty((T, max(top_k, 0)), dtype=torch.int32, device=dev)
    weights = torch.empty((T, max(top_k, 0)), dtype=torch.float32, device=dev)
    plan = None
    if with_plan:
        plan = _empty_plan(T, max(top_k, 0), E, dev)
        workspace = _scratch("nvfp4_moe_route", workspace, lib().nvfp4_moe_workspace_size(T, E, top_k), logits)
    st = lib().nvfp4_moe_route(logits.data_ptr(), _dtype_code(logits.dtype), T, E, ld, _addr(bias), num_groups, group_top_k,
                               top_k, flags, scale, ids.data_ptr(), weights.data_ptr(),
                               plan.offsets.data_ptr() if plan else None, plan.rows.data_ptr() if plan else None,
                               plan.pos.data_ptr() if plan else None, _addr(workspace), _raw_stream(logits))
    _check(st, "nvfp4_moe_route")
    return ids, weights, plan


def nvfp4_moe_route_backward(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor, flags: int = 0,
                             scale: float = 1.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of nvfp4_moe_route's weights with respect to the logits, for the ids it chose."""
    where = "nvfp4_moe_route_backward"
    ld = _matrix(where, "logits", logits)
    T, E = logits.shape
    _want(where, "ids", ids, torch.int32, (T, ids.shape[-1]), logits)
    _want(where, "dweights", dweights, torch.float32, ids.shape, logits)
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError(f"{where}: out must match the logits")
    st = lib().nvfp4_moe_route_backward(logits.data_ptr(), _dtype_code(logits.dtype), T, E, ld, ids.data_ptr(),
                                        dweights.data_ptr(), ids.shape[1], flags, scale, out.data_ptr(),
                                        _matrix(where, "out", out), _raw_stream(logits))
    _check(st, where)
    return out


def nvfp4_moe_plan(ids: torch.Tensor, experts: int, workspace: Optional[torch.Tensor] = None) -> MoEPlan:
    """The plan of a grouped product over ids [tokens, top_k] (int32; ids outside [0, experts) have no
    expert)."""
    if ids.dim() != 2:
        raise ValueError("nvfp4_moe_plan: ids must be 2-D")
    _want("nvfp4_moe_plan", "ids", ids, torch.int32, ids.shape, ids)
    T, k = ids.shape
    plan = _empty_plan(T, k, max(experts, 0), ids.device)
    workspace = _scratch("nvfp4_moe_plan", workspace, lib().nvfp4_moe_workspace_size(T, experts, k), ids)
    st = lib().nvfp4_moe_plan(ids.data_ptr(), T, k, experts, plan.offsets.data_ptr(), plan.rows.data_ptr(),
                              plan.pos.data_ptr(), _addr(workspace), _raw_stream(ids))
    _check(st, "nvfp4_moe_plan")
    return plan


def nvfp4_moe_gather(x: torch.Tensor, plan: MoEPlan, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x[rows / top_k]: the tokens' rows in the plan's order (zero rows where the plan has no slot)."""
    where = "nvfp4_moe_gather"
    ldx = _matrix(where, "x", x)
    T, D = x.shape
    _want(where, "plan.rows", plan.rows, torch.int32, (T * plan.top_k,), x)
    if out is None:
        out = torch.empty((T * plan.top_k, D), dtype=x.dtype, device=x.device)
    elif out.shape != (T * plan.top_k, D) or out.dtype != x.dtype or out.device != x.device:
        raise ValueError(f"{where}: out must be [{T * plan.top_k}, {D}] like x")
    st = lib().nvfp4_moe_gather(x.data_ptr(), _dtype_code(x.dtype), T, D, ldx, plan.rows.data_ptr(), plan.top_k,
                                out.data_ptr(), _matrix(where, "out", out), _raw_stream(x))
    _check(st, where)
    return out


def nvfp4_moe_combine(y: torch.Tensor, plan: MoEPlan, weights: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sum over a token's slots of weight * y[row of the slot] ([tokens * top_k, d] -> [tokens, d]);
    without weights the plain sum, the gradient of nvfp4_moe_gather."""
    where = "nvfp4_moe_combine"
    ldy = _matrix(where, "y", y)
    T, k = plan.pos.shape
    D = y.shape[1]
    if y.shape[0] != T * k:
        raise ValueError(f"{where}: y has {y.shape[0]} rows, the plan {T * k}")
    _want(where, "plan.pos", plan.pos, torch.int32, (T, k), y)
    _want(where, "weights", weights, torch.float32, (T, k), y)
    ldo = D
    if out is None:
        out = torch.empty((T, D), dtype=y.dtype, device=y.device)
    elif out.shape != (T, D) or out.dtype != y.dtype or out.device != y.device:
        raise ValueError(f"{where}: out must be [{T}, {D}] like y")
    else:
        ldo = _matrix(where, "out", out)
    st = lib().nvfp4_moe_combine(y.data_ptr(), _dtype_code(y.dtype), T, D, ldy, plan.pos.data_ptr(), _addr(weights), k,
                                 out.data_ptr(), ldo, _raw_stream(y))
    _check(st, where)
    return out


def nvfp4_moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, plan: MoEPlan, weights: torch.Tensor):
    """Gradients (dy, dweights) of nvfp4_moe_combine with weights."""
    where = "nvfp4_moe_combine_backward"
    ldo, ldy = _matrix(where, "dout", dout), _matrix(where, "y", y)
    T, k = plan.pos.shape
    D = y.shape[1]
    if y.shape[0] != T * k or dout.shape != (T, D) or dout.dtype != y.dtype or dout.device != y.device:
        raise ValueError(f"{where}: dout must be [{T}, {D}] like y [{T * k}, {D}]")
    _want(where, "plan.pos", plan.pos, torch.int32, (T, k), y)
    _want(where, "plan.rows", plan.rows, torch.int32, (T * k,), y)
    _want(where, "weights", weights, torch.float32, (T, k), y)
    dy = torch.empty((T * k, D), dtype=y.dtype, device=y.device)
    dweights = torch.empty((T, k), dtype=torch.float32, device=y.device)
    st = lib().nvfp4_moe_combine_backward(dout.data_ptr(), ldo, y.data_ptr(), ldy, _dtype_code(y.dtype), T, D,
                                          plan.pos.data_ptr(), plan.rows.data_ptr(), weights.data_ptr(), k, dy.data_ptr(), D,
                                          dweights.data_ptr(), _raw_stream(y))
    _check(st, where)
    return dy, dweights


def nvfp4_int8_quantize(x: torch.Tensor, out: Optional[Int8Tensor] = None) -> Int8Tensor:
    """Rows of x (float32 / bfloat16 [rows, cols]) to 8-bit integers with one scale a row."""
    where = "nvfp4_int8_quantize"
    ld = _matrix(where, "x", x)
    R, K = x.shape
    if out is None:
        # (empty_like is the cheapest way to a tensor, and a few tokens' call is mostly that)
        out = Int8Tensor(torch.empty_like(x, dtype=torch.int8, memory_format=torch.contiguous_format),
                         torch.empty(R, dtype=torch.float32, device=x.device), R, K)
    else:
        _want(where, "out.data", out.data, torch.int8, (R, K), x)
        _want(where, "out.scales", out.scales, torch.float32, (R,), x)
    st = lib().nvfp4_int8_quantize(x.data_ptr(), _dtype_code(x.dtype), R, K, ld, out.data.data_ptr(),
                                   out.scales.data_ptr(), _raw_stream(x))
    _check(st, where)
    return out


def nvfp4_int8_gemm(a: Int8Tensor, b: Int8Tensor, out_dtype: torch.dtype = torch.bfloat16, plan: Optional[MoEPlan] = None,
                    gather: bool = False, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = (a * scales) @ (b * scales)^T with exact integer sums.  With a plan: by expert, b holding one
    weight for each; a's rows are in the plan's order, or with gather=True a has one row a token and is
    read through the plan.  Rows of C that the plan gives no expert are not written."""
    where = "nvfp4_int8_gemm"
    if a.k != b.k:
        raise ValueError(f"{where}: a has K={a.k}, b has K={b.k}")
    ad, asc, bd, bsc, n = a.data, a.scales, b.data, b.scales, b.groups * b.rows
    _want(where, "a.data", ad, torch.int8, (a.rows, a.k), ad)
    _want(where, "a.scales", asc, torch.float32, (a.rows,), ad)
    _want(where, "b.data", bd, torch.int8, (n, b.k), ad)
    _want(where, "b.scales", bsc, torch.float32, (n,), ad)
    M, offsets, rows, div = a.rows, None, None, 1
    if plan is not None:
        if plan.experts != b.groups:
            raise ValueError(f"{where}: the plan has {plan.experts} experts, b {b.groups}")
        _want(where, "plan.offsets", plan.offsets, torch.int32, (b.groups + 1,), a.data)
        offsets, M = plan.offsets.data_ptr(), plan.rows.shape[0]
        if gather:
            _want(where, "plan.rows", plan.rows, torch.int32, (a.rows * plan.top_k,), a.data)
            rows, div = plan.rows.data_ptr(), plan.top_k
        elif M != a.rows:
            raise ValueError(f"{where}: a has {a.rows} rows, the plan {M}")
    elif gather or b.groups != 1:
        raise ValueError(f"{where}: a grouped product needs a plan")
    if out is None:
        out = torch.empty((M, b.rows), dtype=out_dtype, device=ad.device)
        ldc = b.rows
    elif out.shape != (M, b.rows) or out.device != ad.device:
        raise ValueError(f"{where}: out must be [{M}, {b.rows}] on {ad.device}")
    else:
        ldc = _matrix(where, "out", out)
    if plan is None:  # (by expert there is none)
        workspace = _scratch(where, workspace, lib().nvfp4_int8_gemm_workspace_size(M, b.rows, b.k), ad)
    st = lib().nvfp4_int8_gemm(ad.data_ptr(), asc.data_ptr(), a.rows, bd.data_ptr(), bsc.data_ptr(), M, b.rows, b.k,
                               out.data_ptr(), _dtype_code(out.dtype), max(ldc, 1), b.groups, offsets, rows, div, _addr(workspace), _raw_stream(ad))
    _check(st, where)
    return out


def _norm_inputs(where, x, y, w_post, gate, w_pre, flags):
    if x.dim() != 2:
        raise ValueError(f"{where}: x must be [tokens, d]")
    T, D = x.shape
    _want(where, "x", x, x.dtype, (T, D), x)
    if y is not None:
        _want(where, "y", y, y.dtype, (T, D), x)
    elif w_post is not None or gate is not None:
        raise ValueError(f"{where}: w_post and gate go with y")
    _want(where, "w_post", w_post, torch.float32, (D,), x)
    _want(where, "w_pre", w_pre, torch.float32, (D,), x)
    if gate is not None and gate.dim() == 2:
        _want(where, "gate", gate, y.dtype, (T, D), x)
        flags |= NVFP4_NORM_TOKEN_GATE
    else:
        _want(where, "gate", gate, torch.float32, (D,), x)
    return T, D, flags


def nvfp4_block_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                     gate: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, alpha: float = 1.0,
                     eps: float = 1e-6, flags: int = 0, n_dtype: Optional[torch.dtype] = None,
                     x_out: Optional[torch.Tensor] = None) -> BlockNorm:
    """x + alpha * gate * norm(y) * w_post and its own norm * w_pre, in one pass (see include/nvfp4.h).
    gate is float32 [d] or [tokens, d] in y's dtype; x_out may be x.  Without y only the second norm (n in
    n_dtype, default x's)."""
    where = "nvfp4_block_norm"
    T, D, flags = _norm_inputs(where, x, y, w_post, gate, w_pre, flags)
    dev = x.device
    y_dtype = y.dtype if y is not None else (n_dtype or x.dtype)
    if y is None:
        if x_out is not None:
            raise ValueError(f"{where}: without y the residual stream does not change")
    elif x_out is None:
        x_out = torch.empty_like(x)
    else:
        _want(where, "x_out", x_out, x.dtype, (T, D), x)
    n = torch.empty_like(x, dtype=y_dtype) if w_pre is not None else None
    rstd = torch.empty((2, T), dtype=torch.float32, device=dev)
    at = rstd.data_ptr()
    st = lib().nvfp4_block_norm(x.data_ptr(), _dtype_code(x.dtype), _addr(y), _dtype_code(y_dtype), T, D, _addr(w_post),
                                _addr(gate), _addr(w_pre), alpha, eps, flags, _addr(x_out), _addr(n), at, at + 4 * T,
                                _raw_stream(x))
    _check(st, where)
    return BlockNorm(x if y is None else x_out, n, rstd, w_post is not None)


def nvfp4_block_norm_backward(dx_out: Optional[torch.Tensor], dn: Optional[torch.Tensor], x: torch.Tensor,
                              y: Optional[torch.Tensor] = None, rstd_post: Optional[torch.Tensor] = None,
                              rstd_pre: Optional[torch.Tensor] = None, w_post: Optional[torch.Tensor] = None,
                              gate: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None, alpha: float = 1.0,
                              flags: int = 0, workspace: Optional[torch.Tensor] = None) -> BlockNormGrads:
    """Gradients of nvfp4_block_norm from dx_out (None: zero) and dn, its inputs (x as it was before the
    call) and its rstd values."""
    where = "nvfp4_block_norm_backward"
    T, D, flags = _norm_inputs(where, x, y, w_post, gate, w_pre, flags)
    dev = x.device
    if (dn is None) != (w_pre is None):
        raise ValueError(f"{where}: dn goes with w_pre")
    y_dtype = y.dtype if y is not None else (dn.dtype if dn is not None else x.dtype)
    _want(where, "dx_out", dx_out, x.dtype, (T, D), x)
    _want(where, "dn", dn, y_dtype, (T, D), x)
    _want(where, "rstd_post", rstd_post, torch.float32, (T,), x)
    _want(where, "rstd_pre", rstd_pre, torch.float32, (T,), x)
    dx = torch.empty_like(x)
    dy = torch.empty_like(y) if y is not None else None
    dw_post = torch.empty(D, dtype=torch.float32, device=dev) if w_post is not None else None
    dgate = torch.empty_like(gate) if gate is not None else None
    dw_pre = torch.empty(D, dtype=torch.float32, device=dev) if w_pre is not None else None
    workspace = _scratch(where, workspace, lib().nvfp4_block_norm_workspace_size(T, D), x)
    st = lib().nvfp4_block_norm_backward(_addr(dx_out), _addr(dn), x.data_ptr(), _dtype_code(x.dtype), _addr(y),
                                         _dtype_code(y_dtype), T, D, _addr(w_post), _addr(gate), _addr(w_pre), alpha, flags,
                                         _addr(rstd_post), _addr(rstd_pre), dx.data_ptr(), _addr(dy), _addr(dw_post),
                                         _addr(dgate), _addr(dw_pre), _addr(workspace), _raw_stream(x))
    _check(st, where)
    return BlockNormGrads(dx, dy, dw_post, dgate, dw_pre)


# ---- fine-tuning beside the quantized products ----------------------------------------------------------
def _enqueue(name: str, like: torch.Tensor, *args):
    """The library's call of this name on the current stream of `like`'s device, with that device current."""
    stream = _raw_stream(like)
    call = getattr(lib(), name)
    if torch._C._cuda_getDevice() == like.device.index:
        st = call(*args, stream)
    else:
        with torch.cuda.device(like.device):
            st = call(*args, stream)
    _check(st, name)


@dataclass
class Adapters:
    """Low-rank factors of `count` adapters, one behind the other (adapters of lower rank are padded with zeros)."""
    a: torch.Tensor       # bfloat16 [count*rank, k]
    b: torch.Tensor       # bfloat16 [count*n, rank]
    scales: torch.Tensor  # float32 [count], of each adapter's product
    rank: int
    k: int
    n: int
    count: int = 1


@dataclass
class AdapterGrads:
    """What nvfp4_adapter_backward gives."""
    dx: torch.Tensor
    da: torch.Tensor  # float32 [count*rank, k]
    db: torch.Tensor  # float32 [count*n, rank]


def _adapter_inputs(where, x, w, plan, gather, by_token):
    """(ldx, M, offsets, rows, pos, row_div, flags) of an adapter's call."""
    bf16, ldx = torch.bfloat16, _matrix(where, "x", x)
    if x.dtype is not bf16:
        raise TypeError(f"{where}: x must be {bf16}, is {x.dtype}")
    if x.shape[1] != w.k:
        raise ValueError(f"{where}: x has K={x.shape[1]}, the adapters K={w.k}")
    _want(where, "w.a", w.a, bf16, (w.count * w.rank, w.k), x)
    _want(where, "w.b", w.b, bf16, (w.count * w.n, w.rank), x)
    _want(where, "w.scales", w.scales, torch.float32, (w.count,), x)
    T = x.shape[0]
    if plan is None:
        if gather or by_token or w.count != 1:
            raise ValueError(f"{where}: more than one adapter needs a plan")
        return ldx, T, None, None, None, 1, 0
    if gather and by_token:
        raise ValueError(f"{where}: rows are gathered or in the tokens' order, not both")
    if plan.experts != w.count:
        raise ValueError(f"{where}: the plan has {plan.experts} adapters, w {w.count}")
    M = plan.rows.shape[0]
    _want(where, "plan.offsets", plan.offsets, torch.int32, (w.count + 1,), x)
    _want(where, "plan.rows", plan.rows, torch.int32, (T * plan.top_k if gather else T,), x)
    if by_token:
        _want(where, "plan.pos", plan.pos, torch.int32, (T, 1), x)
        return ldx, M, plan.offsets.data_ptr(), plan.rows.data_ptr(), plan.pos.data_ptr(), 1, NVFP4_ADAPTER_BY_TOKEN
    return (ldx, M, plan.offsets.data_ptr(), plan.rows.data_ptr(), None, plan.top_k if gather else 1,
            NVFP4_ADAPTER_GATHER if gather else 0)


def _beside(where, name, base, out, shape, dtype, like):
    """(out, its leading dimension, base's) of a call that adds to base."""
    ldb = 0
    if base is not None:
        if base.shape != shape or base.device != like.device:
            raise ValueError(f"{where}: {name} must be {list(shape)} on {like.device}, is {list(base.shape)} on {base.device}")
        ldb, dtype = _matrix(where, name, base), base.dtype
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device), shape[1], ldb
    if out.shape != shape or out.device != like.device or (base is not None and out.dtype is not dtype):
        raise ValueError(f"{where}: out must be {list(shape)} like {name}")
    return out, _matrix(where, "out", out), ldb


def nvfp4_adapter(x: torch.Tensor, w: Adapters, base: Optional[torch.Tensor] = None, plan: Optional[MoEPlan] = None,
                  gather: bool = False, by_token: bool = False, out_dtype: torch.dtype = torch.bfloat16, with_h: bool = False,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """base + scale * (x @ a^T) @ b^T with each row's own adapter (see include/nvfp4.h); returns the result, and with
    with_h=True also h = x @ a^T (float32 [rows, rank], in the plan's order) for the backward call.  plan: of each token's
    adapter (nvfp4_moe_plan of ids [tokens, 1]; by_token=True if x and base are in the tokens' own order) or
    expert (x and base in the plan's order; gather=True if x has one row a token).  Without a plan w is one adapter for
    all rows.  base None: zeros, the result in out_dtype.  out may be base."""
    where = "nvfp4_adapter"
    ldx, M, offsets, rows, pos, div, flags = _adapter_inputs(where, x, w, plan, gather, by_token)
    out, ldc, ldb = _beside(where, "base", base, out, (M, w.n), out_dtype, x)
    h = torch.empty((M, w.rank), dtype=torch.float32, device=x.device) if with_h else None
    workspace = _scratch(where, workspace, lib().nvfp4_adapter_workspace_size(M, w.n, w.k, w.rank, w.count), x)
    _enqueue(where, x, x.data_ptr(), _dtype_code(x.dtype), x.shape[0], max(ldx, w.k), w.a.data_ptr(), w.b.data_ptr(),
             w.scales.data_ptr(), M, w.n, w.k, w.rank, w.count, offsets, rows, pos, div, flags, _addr(base), ldb,
             out.data_ptr(), _dtype_code(out.dtype), ldc, _addr(h), _addr(workspace))
    return (out, h) if with_h else out


def nvfp4_adapter_backward(dout: torch.Tensor, x: torch.Tensor, w: Adapters, h: torch.Tensor,
                           dx_base: Optional[torch.Tensor] = None, plan: Optional[MoEPlan] = None, by_token: bool = False,
                           dx_dtype: torch.dtype = torch.bfloat16, dx: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> AdapterGrads:
    """Gradients of nvfp4_adapter from that of its result (bfloat16), its inputs and its h: dx (added to dx_base, e.g.
    the shared product's own; it may be dx_base) and float32 gradients of the factors.  With gathered rows gather x first."""
    where = "nvfp4_adapter_backward"
    ldx, M, offsets, rows, pos, _, flags = _adapter_inputs(where, x, w, plan, False, by_token)
    if dout.dtype is not torch.bfloat16:
        raise TypeError(f"{where}: dout must be {torch.bfloat16}, is {dout.dtype}")
    if dout.shape != (M, w.n) or dout.device != x.device:
        raise ValueError(f"{where}: dout must be [{M}, {w.n}] on {x.device}")
    _want(where, "h", h, torch.float32, (M, w.rank), x)
    dx, lddx, ldb = _beside(where, "dx_base", dx_base, dx, (M, w.k), dx_dtype, x)
    da = torch.empty((w.count * w.rank, w.k), dtype=torch.float32, device=x.device)
    db = torch.empty((w.count * w.n, w.rank), dtype=torch.float32, device=x.device)
    workspace = _scratch(where, workspace, lib().nvfp4_adapter_backward_workspace_size(M, w.n, w.k, w.rank, w.count), x)
    _enqueue(where, x, dout.data_ptr(), _dtype_code(dout.dtype), _matrix(where, "dout", dout), x.data_ptr(),
             _dtype_code(x.dtype), ldx, w.a.data_ptr(), w.b.data_ptr(), w.scales.data_ptr(), M, w.n, w.k, w.rank, w.count,
             offsets, rows, pos, flags, h.data_ptr(), _addr(dx_base), ldb, dx.data_ptr(), _dtype_code(dx.dtype), lddx,
             da.data_ptr(), db.data_ptr(), _addr(workspace))
    return AdapterGrads(dx, da, db)


@dataclass
class MoEBalance:
    """What nvfp4_moe_balance gives."""
    loss: torch.Tensor    # float32 [1]
    counts: torch.Tensor  # int32 [sequences, experts], slots of each expert
    probs: torch.Tensor   # float32 [sequences, experts], mean probability of each expert
    tokens: torch.Tensor  # int32 [sequences], tokens that have an expert


def nvfp4_moe_balance(logits: torch.Tensor, ids: torch.Tensor, coef: float = 1.0, flags: int = 0, sequences: int = 1,
                      workspace: Optional[torch.Tensor] = None) -> MoEBalance:
    """Balance loss of a routing's ids [tokens, top_k] over its logits [tokens, experts], with the experts' counts, for
    each of `sequences` equal consecutive sequences (see include/nvfp4.h)."""
    where = "nvfp4_moe_balance"
    ld = _matrix(where, "logits", logits)
    T, E = logits.shape
    _want(where, "ids", ids, torch.int32, (T, ids.shape[-1]), logits)
    dev, S = logits.device, max(sequences, 1)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    counts = torch.empty((S, E), dtype=torch.int32, device=dev)
    probs = torch.empty((S, E), dtype=torch.float32, device=dev)
    live = torch.empty(S, dtype=torch.int32, device=dev)
    workspace = _scratch(where, workspace, lib().nvfp4_moe_balance_workspace_size(T, E, sequences), logits)
    _enqueue(where, logits, logits.data_ptr(), _dtype_code(logits.dtype), T, E, ld, ids.data_ptr(), ids.shape[1], sequences, flags,
             coef, loss.data_ptr(), counts.data_ptr(), probs.data_ptr(), live.data_ptr(), _addr(workspace))
    return MoEBalance(loss, counts, probs, live)


def nvfp4_moe_balance_backward(logits: torch.Tensor, ids: torch.Tensor, balance: MoEBalance, coef: float = 1.0, flags: int = 0,
                               dloss: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of nvfp4_moe_balance's loss with respect to the logits, times dloss (float32 [1]; None: 1) and added to
    dlogits (None: 0), e.g. nvfp4_moe_route_backward's result.  out may be dlogits."""
    where = "nvfp4_moe_balance_backward"
    ld = _matrix(where, "logits", logits)
    T, E = logits.shape
    _want(where, "ids", ids, torch.int32, (T, ids.shape[-1]), logits)
    S = balance.counts.shape[0]
    _want(where, "balance.counts", balance.counts, torch.int32, (S, E), logits)
    _want(where, "balance.tokens", balance.tokens, torch.int32, (S,), logits)
    _want(where, "dloss", dloss, torch.float32, (1,), logits)
    for name, t in (("dlogits", dlogits), ("out", out)):
        if t is not None and (t.shape != logits.shape or t.dtype != logits.dtype or t.device != logits.device):
            raise ValueError(f"{where}: {name} must match the logits")
    ld_in = _matrix(where, "dlogits", dlogits) if dlogits is not None else 0
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _enqueue(where, logits, logits.data_ptr(), _dtype_code(logits.dtype), T, E, ld, ids.data_ptr(), ids.shape[1], S, flags, coef,
             balance.counts.data_ptr(), balance.tokens.data_ptr(), _addr(dloss), _addr(dlogits), ld_in, out.data_ptr(),
             _matrix(where, "out", out))
    return out


def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one range of memory, in whatever order of its dimensions."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != step:
            return False
        step *= size
    return True


_DATA_PTR, _NUMEL = torch.Tensor.data_ptr, torch.Tensor.numel
_DEVICE, _CONTIGUOUS = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _host(code: str, values):
    """Host array of these numbers, and its address."""
    a = array.array(code, values)
    return a, a.buffer_info()[0]


def _grad_list(where: str, grads: Sequence[torch.Tensor]):
    """Host arrays of the tensors' addresses, element counts and types, as (arrays, addresses, counts, contiguous): the walk
    over hundreds of tensors is most of a small list's time, so each question is one map over all of them."""
    if isinstance(grads, torch.Tensor) or not len(grads):
        raise ValueError(f"{where}: needs a list of at least one tensor")
    if len(set(map(_DEVICE, grads))) != 1:
        raise ValueError(f"{where}: all tensors must be on one device")
    whole = all(map(_CONTIGUOUS, grads))
    if not whole:
        for t in grads:
            if not _dense(t):
                raise ValueError(f"{where}: a tensor of shape {list(t.shape)} has strides {list(t.stride())}, which leave gaps")
    dtypes = [t.dtype for t in grads]
    codes = {d: _dtype_code(d) for d in set(dtypes)}
    counts = list(map(_NUMEL, grads))
    arrays = (_host("Q", map(_DATA_PTR, grads)), _host("q", counts), _host("i", [codes[d] for d in dtypes]))
    return arrays, counts, dtypes, whole


def _grad_norm(where, grads, listed, flags, workspace):
    (addresses, counts, dtypes), numbers, _, _ = listed
    first, n = grads[0], len(numbers)
    norm = torch.empty(1, dtype=torch.float32, device=first.device)
    workspace = _scratch(where, workspace, lib().nvfp4_grad_workspace_size(n, sum(numbers)), first)
    _enqueue("nvfp4_grad_norm", first, addresses[1], counts[1], dtypes[1], n, flags, norm.data_ptr(), _addr(workspace))
    return norm


def nvfp4_grad_norm(grads: Sequence[torch.Tensor], flags: int = 0, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Norm (float32 [1]) of all tensors of the list together (float32 / bfloat16, in any mixture): the square root of
    the sum of squares, or with NVFP4_GRAD_MAX the largest magnitude."""
    where = "nvfp4_grad_norm"
    return _grad_norm(where, grads, _grad_list(where, grads), flags, workspace)


def nvfp4_grad_clip(grads: Sequence[torch.Tensor], max_norm: float, flags: int = 0, eps: float = 1e-6,
                    out: Optional[Sequence[torch.Tensor]] = None, norm: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale the tensors of the list, in place or into out, by min(1, max_norm / (norm + eps)); returns the norm
    (float32 [1]), which is that of the list unless it is given (e.g. that of all ranks).  A norm that is infinite or NaN
    leaves the gradients as they are."""
    where = "nvfp4_grad_clip"
    listed = _grad_list(where, grads)
    (addresses, counts, dtypes), numbers, types, whole = listed
    outs = addresses
    if out is not None:
        # (contiguous tensors are a row of elements, whatever their shapes)
        if len(out) != len(numbers) or list(map(_NUMEL, out)) != numbers or [o.dtype for o in out] != types or \
                set(map(_DEVICE, out)) != {grads[0].get_device()} or \
                not (whole and all(map(_CONTIGUOUS, out)) or
                     all(o.shape == t.shape and o.stride() == t.stride() for o, t in zip(out, grads))):
            raise ValueError(f"{where}: out must match the list, tensor by tensor")
        outs = _host("Q", map(_DATA_PTR, out))
    _want(where, "norm", norm, torch.float32, (1,), grads[0])
    if norm is None:
        norm = _grad_norm(where, grads, listed, flags, workspace)
    _enqueue(where, grads[0], addresses[1], outs[1], counts[1], dtypes[1], len(numbers), norm.data_ptr(), max_norm, eps)
    return norm
