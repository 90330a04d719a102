"""ctypes binding of libtg (include/tg.h).  Argument marshalling only.

Every compute step runs in the CUDA kernels of libtg.so.  There is no Python,
PyTorch or CPU fallback: if the library is not built, or the device is not a
GB300 (sm_103a), these functions raise.  PyTorch supplies device memory and
streams; tensors are passed as raw device pointers with their strides.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# TG_LIB_PATH selects another build of the library (e.g. to compare two builds on one GPU).
LIB_PATH = os.environ.get("TG_LIB_PATH") or os.path.join(_PKG, "libtg.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "tg.h")

TG_OK, TG_ERR_INVALID_ARG, TG_ERR_UNSUPPORTED, TG_ERR_CUDA, TG_ERR_TIMEOUT, TG_ERR_NO_DEVICE = range(6)
STATUS_NAMES = {0: "TG_OK", 1: "TG_ERR_INVALID_ARG", 2: "TG_ERR_UNSUPPORTED", 3: "TG_ERR_CUDA",
                4: "TG_ERR_TIMEOUT", 5: "TG_ERR_NO_DEVICE"}
EPILOGUES = {"none": 0, "bias": 1, "bias_gelu": 2}
ROW_MAJOR, COL_MAJOR = 0, 1
BF16, F32, F16, E4M3, E5M2 = 0, 1, 2, 3, 4
_DTYPE_CODE = {torch.bfloat16: BF16, torch.float32: F32, torch.float16: F16}
_FP8_CODE = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
FP8_BLOCK = 128     # values that share a scale
_ITEM_BYTES = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4, torch.float8_e4m3fn: 1, torch.float8_e5m2: 1}

_lib = None
_lock = threading.Lock()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class TGError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


class GroupProblem(ctypes.Structure):
    """Mirror of tg_group_problem (field order and natural alignment as in tg.h)."""
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("layout_a", ctypes.c_int),
        ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("layout_b", ctypes.c_int),
        ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("c_dtype", ctypes.c_int),
        ("epi", ctypes.c_int),
        ("bias", ctypes.c_void_p),
        ("ab_dtype", ctypes.c_int),
    ]


class Fp8Operand(ctypes.Structure):
    """Mirror of tg_scaled_operand."""
    _fields_ = [
        ("data", ctypes.c_void_p), ("ld", ctypes.c_int64),
        ("scale", ctypes.c_void_p), ("scale_stride", ctypes.c_int64), ("scale_k_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int), ("layout", ctypes.c_int), ("block", ctypes.c_int),
    ]


def header_functions() -> list[str]:
    """Names of the functions include/tg.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tg_[a-z_]+)\s*\(", text)))


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libtg.so (built by grouped_gemm_persistent_gb300.build); raise if it is missing."""
    global _lib
    if path is None and _lib is not None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libtg.so is not built ({p}); run `python -m grouped_gemm_persistent_gb300.build`")
        lib = ctypes.CDLL(p)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        lib.tg_gemm.restype = ci
        lib.tg_gemm.argtypes = [vp, ci, i64, vp, ci, i64, vp, ci, i64, i64, i64, i64, ci, vp, vp]
        lib.tg_gemm_ex.restype = ci
        lib.tg_gemm_ex.argtypes = [ctypes.POINTER(GroupProblem), vp]
        lib.tg_gemm_bcast.restype = ci
        lib.tg_gemm_bcast.argtypes = [vp, ci, i64, i64, i64, vp, ci, i64, vp, ci, i64, i64, i64, ci, vp, vp]
        lib.tg_moe_gemm.restype = ci
        lib.tg_moe_gemm.argtypes = [vp, i64, i64, i64, vp, ci, i64, i64, i64, i64, vp, ci, i64, vp, ci, vp, vp]
        lib.tg_row_rms.restype = ci
        lib.tg_row_rms.argtypes = [vp, i64, i64, i64, ctypes.c_float, vp, vp]
        lib.tg_gemm_rmsnorm.restype = ci
        lib.tg_gemm_rmsnorm.argtypes = [vp, i64, vp, ci, i64, vp, ci, i64, i64, i64, i64, ctypes.c_float, vp, ci,
                                        vp, vp]
        lib.tg_grouped_gemm.restype = ci
        lib.tg_grouped_gemm.argtypes = [ctypes.POINTER(GroupProblem), ci, vp]
        lib.tg_grouped_gemm_noalloc.restype = ci
        lib.tg_grouped_gemm_noalloc.argtypes = [ctypes.POINTER(GroupProblem), ci, vp]
        lib.tg_quantize_blocks.restype = ci
        lib.tg_quantize_blocks.argtypes = [vp, ci, i64, i64, i64, ci, ci, vp, ci, i64, vp, i64, vp]
        op8 = ctypes.POINTER(Fp8Operand)
        lib.tg_gemm_scaled.restype = ci
        lib.tg_gemm_scaled.argtypes = [op8, op8, vp, ci, i64, i64, i64, i64, ci, vp, vp]
        lib.tg_moe_gemm_scaled.restype = ci
        lib.tg_moe_gemm_scaled.argtypes = [op8, i64, i64, op8, i64, i64, i64, i64, vp, ci, i64, vp, ci, vp, vp]
        lib.tg_moe_router.restype = ci
        lib.tg_moe_router.argtypes = [vp, ci, i64, i64, i64, i64, ci, vp, vp, vp, vp, vp, vp]
        lib.tg_moe_router_backward.restype = ci
        lib.tg_moe_router_backward.argtypes = [vp, ci, i64, i64, i64, i64, ci, vp, vp, vp, vp, vp, vp, i64, vp]
        lib.tg_rmsnorm.restype = ci
        lib.tg_rmsnorm.argtypes = [ctypes.c_char_p, vp]
        lib.tg_rmsnorm_backward.restype = ci
        lib.tg_rmsnorm_backward.argtypes = [ctypes.c_char_p, vp]
        lib.tg_moe_router_scored.restype = ci
        lib.tg_moe_router_scored.argtypes = [ctypes.c_char_p, vp]
        lib.tg_moe_router_scored_backward.restype = ci
        lib.tg_moe_router_scored_backward.argtypes = [ctypes.c_char_p, vp]
        lib.tg_lora_add.restype = ci
        lib.tg_lora_add.argtypes = [ctypes.c_char_p, vp]
        lib.tg_status_string.restype = ctypes.c_char_p
        lib.tg_status_string.argtypes = [ci]
        lib.tg_last_error_message.restype = ctypes.c_char_p
        lib.tg_last_error_message.argtypes = []
        lib.tg_device_status.restype = ci
        lib.tg_device_status.argtypes = [vp]
        lib.tg_set_wait_budget_ms.restype = ci
        lib.tg_set_wait_budget_ms.argtypes = [ctypes.c_uint32]
        lib.tg_debug_withhold_stage.restype = ci
        lib.tg_debug_withhold_stage.argtypes = [i64]
        lib.tg_debug_withhold_stage_in.restype = ci
        lib.tg_debug_withhold_stage_in.argtypes = [i64, ctypes.c_int32]
        lib.tg_debug_trace.restype = ci
        lib.tg_debug_trace.argtypes = [vp, i64, vp, i64]
        lib.tg_version.restype = ctypes.c_uint32
        lib.tg_version.argtypes = []
        lib.tg_launch_count.restype = ctypes.c_uint64
        lib.tg_launch_count.argtypes = []
        if path is None:
            _lib = lib
        return lib


def _check(status: int) -> None:
    if status != TG_OK:
        msg = load().tg_last_error_message().decode(errors="replace")
        raise TGError(status, msg)


def _stream_handle(stream) -> int:
    if stream is None:
        if _raw_stream is not None:      # the handle alone, without the Stream object around it
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _matrix(t: torch.Tensor, name: str):
    """(layout, ld) of a 2-D tensor view: row-major if its rows are contiguous, else column-major.

    With a single row (or column) the leading dimension is never used to step;
    it is then reported as the extent rounded up to 8 elements, which keeps the
    TMA stride rule satisfied.
    """
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    r, c = t.shape
    s0, s1 = t.stride()
    if s1 == 1 or c == 1:
        return ROW_MAJOR, (s0 if r > 1 else -(-max(c, 1) // 8) * 8)
    if s0 == 1 or r == 1:
        return COL_MAJOR, (s1 if c > 1 else -(-max(r, 1) // 8) * 8)
    raise ValueError(f"{name}: neither rows nor columns are contiguous (strides {t.stride()})")


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def gemm(a: torch.Tensor, b: torch.Tensor, out: torch.Tensor | None = None, *, bias: torch.Tensor | None = None,
         epilogue: str = "none", out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """out[M,N] = epilogue(a[M,K] @ b[K,N]) on the GPU (tg_gemm, or tg_gemm_ex for fp16 operands).

    ``a``/``b`` are bf16 or fp16 CUDA tensors of the same type (``bias`` too);
    each may be a row-major or column-major view (a transposed view of a
    row-major tensor is column-major).  ``out`` (bf16, fp16 or fp32, rows
    contiguous, row stride may exceed N) is allocated if not given.
    Asynchronous on ``stream`` (default: torch's current stream).
    """
    if a.dtype not in (torch.bfloat16, torch.float16) or b.dtype != a.dtype:
        raise TypeError("a and b must both be torch.bfloat16 or both torch.float16")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if out.dtype not in _DTYPE_CODE or tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N] bf16, fp16 or fp32")
    la, lda = _matrix(a, "a")
    lb, ldb = _matrix(b, "b")
    lc, ldc = _matrix(out, "out")
    if lc != ROW_MAJOR:
        raise ValueError("out must be row-major")
    epi = EPILOGUES[epilogue]
    if epi and (bias is None or bias.dtype != a.dtype or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError("this epilogue needs a contiguous bias of length N with the operands' dtype")
    if a.dtype == torch.bfloat16:
        _check(load().tg_gemm(_ptr(a), la, lda, _ptr(b), lb, ldb, _ptr(out), _DTYPE_CODE[out.dtype], ldc, M, N, K,
                              epi, _ptr(bias) if epi else None, _stream_handle(stream)))
    else:
        prob = GroupProblem(M, N, K, _ptr(a), lda, la, _ptr(b), ldb, lb, _ptr(out), ldc, _DTYPE_CODE[out.dtype], epi,
                            _ptr(bias) if epi else None, F16)
        _check(load().tg_gemm_ex(ctypes.byref(prob), _stream_handle(stream)))
    return out


def gemm_bcast(a_user: torch.Tensor, b: torch.Tensor, repeat: int, out: torch.Tensor | None = None, *,
               bias: torch.Tensor | None = None, epilogue: str = "none", out_dtype: torch.dtype = torch.bfloat16,
               stream=None) -> torch.Tensor:
    """out[U*repeat, N] = epilogue(A @ b) with A's row i*repeat + j equal to a_user[i] (tg_gemm_bcast).

    The repeated rows are never materialised: the kernel reads ``a_user`` [U, K]
    once per replica and stores each result row ``repeat`` times.
    """
    if a_user.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise TypeError("a_user and b must be torch.bfloat16")
    U, K = a_user.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((U * repeat, N), dtype=out_dtype, device=a_user.device)
    if tuple(out.shape) != (U * repeat, N):
        raise ValueError("out must be [U * repeat, N]")
    la, lda = _matrix(a_user, "a_user")
    lb, ldb = _matrix(b, "b")
    lc, ldc = _matrix(out, "out")
    if lc != ROW_MAJOR:
        raise ValueError("out must be row-major")
    epi = EPILOGUES[epilogue]
    if epi and (bias is None or bias.dtype != torch.bfloat16 or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError("this epilogue needs a contiguous bf16 bias of length N")
    _check(load().tg_gemm_bcast(_ptr(a_user), la, lda, U, repeat, _ptr(b), lb, ldb, _ptr(out),
                                _DTYPE_CODE[out.dtype], ldc, N, K, epi,
                                _ptr(bias) if epi else None, _stream_handle(stream)))
    return out


def _row_major_bf16(a: torch.Tensor, name: str) -> int:
    if a.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16")
    la, lda = _matrix(a, name)
    if la != ROW_MAJOR:
        raise ValueError(f"{name} must be row-major")
    return lda


def row_rms(a: torch.Tensor, eps: float, out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """out[i] = 1 / sqrt(mean_k a[i, k]^2 + eps), fp32 [M], for a row-major bf16 ``a`` (tg_row_rms)."""
    lda = _row_major_bf16(a, "a")
    M, K = a.shape
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=a.device)
    if out.dtype != torch.float32 or out.numel() != M or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 tensor of length M")
    _check(load().tg_row_rms(_ptr(a), lda, M, K, float(eps), _ptr(out), _stream_handle(stream)))
    return out


def gemm_rmsnorm(a: torch.Tensor, b: torch.Tensor, eps: float, out: torch.Tensor | None = None, *,
                 row_scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, epilogue: str = "none",
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """out = epilogue(rmsnorm(a) @ b) with the normalisation fused into the GEMM (tg_gemm_rmsnorm).

    ``a`` is row-major bf16 [M, K]; ``b`` bf16 [K, N] in either layout.  The row
    factors land in ``row_scale`` (fp32 [M], allocated if not given).
    """
    lda = _row_major_bf16(a, "a")
    if b.dtype != torch.bfloat16:
        raise TypeError("b must be torch.bfloat16")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
    if out.dtype not in _DTYPE_CODE or tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N] bf16, fp16 or fp32")
    if row_scale is None:
        row_scale = torch.empty(M, dtype=torch.float32, device=a.device)
    if row_scale.dtype != torch.float32 or row_scale.numel() != M or not row_scale.is_contiguous():
        raise ValueError("row_scale must be a contiguous fp32 tensor of length M")
    lb, ldb = _matrix(b, "b")
    lc, ldc = _matrix(out, "out")
    if lc != ROW_MAJOR:
        raise ValueError("out must be row-major")
    epi = EPILOGUES[epilogue]
    if epi and (bias is None or bias.dtype != torch.bfloat16 or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError("this epilogue needs a contiguous bf16 bias of length N")
    _check(load().tg_gemm_rmsnorm(_ptr(a), lda, _ptr(b), lb, ldb, _ptr(out), _DTYPE_CODE[out.dtype], ldc, M, N, K,
                                  float(eps), _ptr(row_scale), epi, _ptr(bias) if epi else None,
                                  _stream_handle(stream)))
    return out


def moe_gemm_device(a: torch.Tensor, b: torch.Tensor, counts: torch.Tensor, out: torch.Tensor | None = None, *,
                    bias: torch.Tensor | None = None, epilogue: str = "none",
                    out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """MoE expert GEMM with the token counts on the GPU (tg_moe_gemm): no host round trip.

    ``a`` [T, K] bf16 row-major, rows grouped by expert; ``b`` [G, K, N] bf16 with
    each expert row-major (``b[g]`` contiguous rows) or column-major (a view of
    a [G, N, K] tensor); ``counts`` int32 CUDA tensor [G]; ``out`` [T, N]; rows
    past sum(counts) are not written.  ``bias`` is [G, N] bf16.
    """
    if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise TypeError("a and b must be torch.bfloat16")
    if counts.dtype != torch.int32 or not counts.is_cuda or counts.dim() != 1 or not counts.is_contiguous():
        raise TypeError("counts must be a contiguous int32 CUDA tensor [G]")
    T, K = a.shape
    G, K2, N = b.shape
    if K != K2 or counts.shape[0] != G:
        raise ValueError("shapes: a [T, K], b [G, K, N], counts [G]")
    la, lda = _matrix(a, "a")
    if la != ROW_MAJOR:
        raise ValueError("a must be row-major")
    if b.stride(2) == 1:
        lb, ldb = ROW_MAJOR, b.stride(1)
    elif b.stride(1) == 1:
        lb, ldb = COL_MAJOR, b.stride(2)
    else:
        raise ValueError("each expert of b must be row- or column-major")
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype, device=a.device)
    lc, ldc = _matrix(out, "out")
    epi = EPILOGUES[epilogue]
    if epi and (bias is None or bias.dtype != torch.bfloat16 or tuple(bias.shape) != (G, N) or not bias.is_contiguous()):
        raise ValueError("this epilogue needs a contiguous bf16 bias [G, N]")
    _check(load().tg_moe_gemm(_ptr(a), lda, T, K, _ptr(b), lb, ldb, b.stride(0), G, N, _ptr(out),
                              _DTYPE_CODE[out.dtype], ldc, counts.data_ptr(), epi, _ptr(bias) if epi else None,
                              _stream_handle(stream)))
    return out


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _stream_object(stream, device) -> torch.cuda.Stream:
    """The torch stream whose order a handle's work follows."""
    handle = _stream_handle(stream)
    # NULL, cudaStreamLegacy, and cudaStreamPerThread, which waits for the legacy stream's work and is waited for by it
    if handle in (0, 1, 2):
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _empty(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """An uninitialised tensor on ``like``'s device, in the allocator's order of ``stream`` (an object or a raw
    handle), so that a block freed on another stream is not handed out while that stream still uses it."""
    if stream is None or not like.is_cuda:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = _stream_object(stream, like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rows_of_16_bytes(like: torch.Tensor, rows: int, cols: int, dtype: torch.dtype, stream) -> tuple[torch.Tensor, int]:
    """An uninitialised [rows, cols] tensor whose rows start on 16-byte boundaries, and its leading dimension."""
    step = 16 // _ITEM_BYTES[dtype]
    ld = -(-cols // step) * step
    t = _empty(like, (rows, ld), dtype, stream)
    return (t if ld == cols else t[:, :cols]), max(ld, 1)


def _on_one_gpu(names: str, *tensors) -> None:
    """The tensors (None is left out) are on one CUDA device, the current one."""
    current = torch.cuda.current_device() if tensors[0].is_cuda else -1
    for i, t in enumerate(tensors):
        if t is not None and (t.get_device() != current or current < 0):
            raise ValueError(f"{names.split()[i]} must be on the current CUDA device, got {t.device}")


def _row_major_ld(t: torch.Tensor, name: str, cols: int) -> int:
    """Leading dimension of a row-major matrix of `cols` columns (a single row's is never stepped by)."""
    s0, s1 = t.stride()
    if s1 == 1 or cols <= 1:
        return s0 if t.shape[0] > 1 else max(cols, 1)
    raise ValueError(f"{name} must be row-major (strides {t.stride()})")


def quantize_fp8(x: torch.Tensor, block: tuple[int, int] = (1, 128), q: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, *, dtype: torch.dtype = torch.float8_e4m3fn,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): ``x`` [M, K] in 8 bits with one power-of-two scale for each ``block`` of values (tg_quantize_blocks).

    ``block`` is (1, 128), (128, 1) or (128, 128); ``scale`` (fp32) is [M, ceil(K / 128)] (a transposed view:
    a block column's scales lie side by side), [ceil(M / 128), K] or [ceil(M / 128), ceil(K / 128)].  ``x`` is
    row-major bf16, fp16 or fp32; ``q`` (allocated with rows of a multiple of 16 bytes if not given) has
    ``dtype`` torch.float8_e4m3fn or torch.float8_e5m2, and ``x`` is ``q * scale`` up to its rounding.
    """
    xt = _DTYPE_CODE.get(x.dtype)
    if xt is None:
        raise TypeError("x must be bf16, fp16 or fp32")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    M, K = x.shape
    ldx = _row_major_ld(x, "x", K)
    br, bc = block
    by_row = br == 1
    if (br, bc) not in ((1, 128), (128, 1), (128, 128)):
        raise ValueError(f"block must be (1, 128), (128, 1) or (128, 128), got {block}")
    rows, cols = M if by_row else (M + 127) // 128, K if bc == 1 else (K + 127) // 128     # of the scales
    if q is None:
        if dtype not in _FP8_CODE:
            raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
        q, ldq = _rows_of_16_bytes(x, M, K, dtype, stream)
    else:
        dtype = q.dtype
        if dtype not in _FP8_CODE or q.shape != x.shape:
            raise ValueError("q must be [M, K] float8_e4m3fn or float8_e5m2")
        ldq = _row_major_ld(q, "q", K)
    if scale is None:
        # a row's scales are the columns of the result: a block column's lie side by side
        stored = _empty(x, (cols, rows) if by_row else (rows, cols), torch.float32, stream)
        scale, scale_ld = (stored.t() if by_row else stored), max(rows if by_row else cols, 1)
    else:
        if scale.dtype != torch.float32 or tuple(scale.shape) != (rows, cols):
            raise ValueError(f"scale must be fp32 {[rows, cols]}")
        (inner, outer), (si, so) = ((rows, cols), scale.stride()) if by_row else ((cols, rows), scale.stride()[::-1])
        if inner > 1 and si != 1:
            raise ValueError("scale must have " + ("contiguous columns" if by_row else "contiguous rows"))
        scale_ld = so if outer > 1 else max(inner, 1)
    _on_one_gpu("x q scale", x, q, scale)
    status = load().tg_quantize_blocks(x.data_ptr(), xt, ldx, M, K, br, bc, q.data_ptr(), _FP8_CODE[dtype], ldq,
                                       scale.data_ptr(), scale_ld, _stream_handle(stream))
    if status:
        _check(status)
    return q, scale


def _fp8_layout(r: int, c: int, s0: int, s1: int, name: str) -> tuple[int, int]:
    """(layout, ld) of an r x c matrix with strides (s0, s1).  A single row or column is never stepped past: its
    leading dimension is reported as its extent rounded up to 16 elements."""
    if s1 == 1 and (c != 1 or r <= 1):
        return ROW_MAJOR, (s0 if r > 1 else -(-max(c, 1) // 16) * 16)
    if s0 == 1:
        return COL_MAJOR, (s1 if c > 1 else -(-max(r, 1) // 16) * 16)
    if c == 1:
        return ROW_MAJOR, s0
    if r == 1:
        return COL_MAJOR, s1
    raise ValueError(f"{name}: neither rows nor columns are contiguous (strides {(s0, s1)})")


def _fp8_matrix(t: torch.Tensor, name: str) -> tuple[int, int]:
    """(layout, ld) of a 2-D 8-bit tensor view."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return _fp8_layout(*t.shape, *t.stride(), name)


def _bad_scale(s: torch.Tensor, name: str, rows: int, kb: int):
    return ValueError(f"{name} must be fp32 with {kb} blocks of K and {rows} or {_blocks(rows)} entries, "
                      f"got {tuple(s.shape)} {s.dtype}")


def _fp8_types(a: torch.Tensor, b: torch.Tensor) -> tuple[int, int]:
    ta, tb = _FP8_CODE.get(a.dtype), _FP8_CODE.get(b.dtype)
    if ta is None or tb is None:
        raise TypeError("a and b must be float8_e4m3fn or float8_e5m2")
    return ta, tb


def gemm_fp8(a: torch.Tensor, scale_a: torch.Tensor, b: torch.Tensor, scale_b: torch.Tensor,
             out: torch.Tensor | None = None, *, bias: torch.Tensor | None = None, epilogue: str = "none",
             out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """out[M,N] = epilogue((a * scale_a) @ (b * scale_b)) for 8-bit operands with a scale per block of 128 (tg_gemm_scaled).

    ``a`` [M, K] and ``b`` [K, N] are float8_e4m3fn or float8_e5m2, each a row-major or column-major view.
    ``scale_a`` is fp32 [M, ceil(K / 128)] (or [ceil(M / 128), ...]), ``scale_b`` [ceil(K / 128), N] or
    [ceil(K / 128), ceil(N / 128)], with any strides; scales of which neighbouring rows lie side by side
    (quantize_fp8's) load fastest.  ``bias`` is bf16 [N]; ``out`` is bf16, fp16 or fp32 (allocated if not given, its rows
    on 16-byte boundaries: a view with a wider row stride where N is not a multiple of 16 bytes).
    """
    ta, tb = _fp8_types(a, b)
    la, lda = _fp8_matrix(a, "a")
    lb, ldb = _fp8_matrix(b, "b")
    M, K = a.shape
    K2, N = b.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    kb = (K + 127) // 128
    if scale_a.dtype != torch.float32 or scale_a.dim() != 2:
        raise _bad_scale(scale_a, "scale_a", M, kb)
    rows, cols = scale_a.shape
    if cols != kb or (rows != M and rows != (M + 127) // 128):
        raise _bad_scale(scale_a, "scale_a", M, kb)
    sa, sak = scale_a.stride()
    ba = 1 if rows == M else 128
    if scale_b.dtype != torch.float32 or scale_b.dim() != 2:
        raise _bad_scale(scale_b, "scale_b", N, kb)
    rows, cols = scale_b.shape
    if rows != kb or (cols != N and cols != (N + 127) // 128):
        raise _bad_scale(scale_b, "scale_b", N, kb)
    sbk, sb = scale_b.stride()
    bb = 1 if cols == N else 128
    if out is None:
        ct = _DTYPE_CODE.get(out_dtype)
        if ct is None:
            raise TypeError("out_dtype must be bf16, fp16 or fp32")
        out, ldc = _rows_of_16_bytes(a, M, N, out_dtype, stream)
    else:
        ct = _DTYPE_CODE.get(out.dtype)
        if ct is None or tuple(out.shape) != (M, N):
            raise ValueError("out must be [M, N] bf16, fp16 or fp32")
        ldc = _row_major_ld(out, "out", N)
    epi = EPILOGUES[epilogue]
    if not epi:
        bias = None
    elif bias is None or bias.dtype != torch.bfloat16 or bias.numel() != N or not bias.is_contiguous():
        raise ValueError("this epilogue needs a contiguous bf16 bias of length N")
    _on_one_gpu("a scale_a b scale_b out bias", a, scale_a, b, scale_b, out, bias)
    oa = Fp8Operand(a.data_ptr(), lda, scale_a.data_ptr(), sa, sak, ta, la, ba)
    ob = Fp8Operand(b.data_ptr(), ldb, scale_b.data_ptr(), sb, sbk, tb, lb, bb)
    status = load().tg_gemm_scaled(oa, ob, out.data_ptr(), ct, ldc, M, N, K, epi, bias.data_ptr() if epi else None,
                                   _stream_handle(stream))
    if status:
        _check(status)
    return out


def moe_gemm_fp8(a: torch.Tensor, scale_a: torch.Tensor, b: torch.Tensor, scale_b: torch.Tensor, counts: torch.Tensor,
                 out: torch.Tensor | None = None, *, bias: torch.Tensor | None = None, epilogue: str = "none",
                 out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """moe_gemm_device with 8-bit operands (tg_moe_gemm_scaled): the token counts stay on the GPU.

    ``a`` [T, K] row-major, rows grouped by expert, ``scale_a`` [T, ceil(K / 128)]; ``b`` [G, K, N], each expert
    row- or column-major, ``scale_b`` [G, ceil(K / 128), ceil(N / 128)]; ``counts`` int32 CUDA tensor [G];
    ``out`` [T, N], rows past sum(counts) not written; ``bias`` bf16 [G, N].
    """
    ta, tb = _fp8_types(a, b)
    if counts.dtype != torch.int32 or counts.dim() != 1 or not counts.is_contiguous():
        raise TypeError("counts must be a contiguous int32 tensor [G]")
    la, lda = _fp8_matrix(a, "a")
    if la != ROW_MAJOR:
        raise ValueError("a must be row-major")
    T, K = a.shape
    if b.dim() != 3 or b.shape[1] != K or counts.shape[0] != b.shape[0]:
        raise ValueError("shapes: a [T, K], b [G, K, N], counts [G]")
    G, _, N = b.shape
    kb = (K + 127) // 128
    if scale_a.dtype != torch.float32 or tuple(scale_a.shape) != (T, kb):
        raise ValueError(f"scale_a must be fp32 {[T, kb]}")
    if scale_b.dtype != torch.float32 or tuple(scale_b.shape) != (G, kb, (N + 127) // 128):
        raise ValueError(f"scale_b must be fp32 {[G, kb, (N + 127) // 128]}")
    if out is None:
        ct = _DTYPE_CODE.get(out_dtype)
        if ct is None:
            raise TypeError("out_dtype must be bf16, fp16 or fp32")
        out, ldc = _rows_of_16_bytes(a, T, N, out_dtype, stream)
    else:
        ct = _DTYPE_CODE.get(out.dtype)
        if ct is None or tuple(out.shape) != (T, N):
            raise ValueError("out must be [T, N] bf16, fp16 or fp32")
        ldc = _row_major_ld(out, "out", N)
    epi = EPILOGUES[epilogue]
    if not epi:
        bias = None
    elif bias is None or bias.dtype != torch.bfloat16 or tuple(bias.shape) != (G, N) or not bias.is_contiguous():
        raise ValueError("this epilogue needs a contiguous bf16 bias [G, N]")
    _on_one_gpu("a scale_a b scale_b counts out bias", a, scale_a, b, scale_b, counts, out, bias)
    if G == 0:
        return out
    expert, s0, s1 = b.stride()
    lb, ldb = _fp8_layout(K, N, s0, s1, "b")
    if G == 1:
        expert = (K if lb == ROW_MAJOR else N) * ldb
    sg, sbk, sb = scale_b.stride()
    sa, sak = scale_a.stride()
    oa = Fp8Operand(a.data_ptr(), lda, scale_a.data_ptr(), sa, sak, ta, la, 1)
    ob = Fp8Operand(b.data_ptr(), ldb, scale_b.data_ptr(), sb, sbk, tb, lb, 128)
    status = load().tg_moe_gemm_scaled(oa, T, K, ob, expert, sg, G, N, out.data_ptr(), ct, ldc, counts.data_ptr(), epi,
                                       bias.data_ptr() if epi else None, _stream_handle(stream))
    if status:
        _check(status)
    return out


# Records of arguments, packed straight into bytes: quicker than a ctypes structure or twenty converted arguments.
_RMSNORM = struct.Struct("@qq" + 2 * "Qq" + "Q" + 4 * "Qq" + "Q" + "f5i")                    # tg_rmsnorm_args
_RMSNORM_BACKWARD = struct.Struct("@qq" + 2 * "Qq" + "QQ" + 2 * "Qq" + "Q" + "3i4x")         # tg_rmsnorm_backward_args

_ROUTER = struct.Struct("@3q" + "Qq" + "Q" + "3q" + "5Q" + "f3i")                            # tg_router_args
_ROUTER_BACKWARD = struct.Struct("@3q" + "Qq" + "4Q" + "Qq" + "f3i")                         # tg_router_backward_args
_LORA = struct.Struct("@5q" + "Qq" + 2 * "Qqq" + "QQ" + 2 * "Qq" + "2i")                     # tg_lora_args
SCORES = {"softmax": 0, "sigmoid": 1}


class Normed(NamedTuple):
    """What rmsnorm returns, and rmsnorm_backward needs again."""
    y: torch.Tensor | None        # the normalised rows
    q: torch.Tensor | None        # their 8-bit copy
    scale: torch.Tensor | None    # its scales
    hidden: torch.Tensor          # x + residual (x itself without one)
    row_scale: torch.Tensor       # fp32 [M], 1 / rms


def _rows_like(t: torch.Tensor, name: str, like: torch.Tensor) -> int:
    """Leading dimension of a row-major tensor of another's shape."""
    if t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}, got {list(t.shape)}")
    return _row_major_ld(t, name, like.shape[1])


def _gain(gain: torch.Tensor | None, K: int) -> tuple[int, int]:
    """(pointer, type code) of a gain vector."""
    if gain is None:
        return 0, 0
    code = _DTYPE_CODE.get(gain.dtype)
    if code is None:
        raise TypeError("gain must be bf16, fp16 or fp32")
    if gain.shape != (K,) or (K > 1 and gain.stride(0) != 1):
        raise ValueError(f"gain must be a contiguous vector of length {K}")
    return gain.data_ptr(), code


def rmsnorm(x: torch.Tensor, gain: torch.Tensor | None = None, eps: float = 1e-6, *,
            residual: torch.Tensor | None = None, hidden: torch.Tensor | None = None,
            out_dtype: torch.dtype | None = torch.bfloat16, fp8_dtype: torch.dtype | None = None,
            stream=None) -> Normed:
    """RMS norm of the rows of ``x + residual``, in ``out_dtype`` and / or in 8 bits (tg_rmsnorm).

    ``x`` [M, K] is row-major bf16, fp16 or fp32, ``residual`` (None: x alone) of x's type or fp32; their sum, rounded
    to the residual's type, is the result's ``hidden`` (written to ``hidden`` if given, which may be the residual).
    ``gain`` [K] is bf16, fp16 or fp32.  ``y`` is ``hidden / rms * gain`` in ``out_dtype`` (None: not wanted);
    with ``fp8_dtype`` (torch.float8_e4m3fn or torch.float8_e5m2) ``q`` and ``scale`` are what
    ``quantize_fp8(y, (1, 128))`` makes of the fp32 y: the operands of gemm_fp8 and moe_gemm_fp8.
    """
    xt = _DTYPE_CODE.get(x.dtype)
    if xt is None:
        raise TypeError("x must be bf16, fp16 or fp32")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    M, K = x.shape
    ldx = _row_major_ld(x, "x", K)
    rt = ldr = ldh = 0
    if residual is not None:
        if residual.dtype != x.dtype and residual.dtype != torch.float32:
            raise TypeError("residual must have x's type or fp32")
        rt = _DTYPE_CODE[residual.dtype]
        ldr = _rows_like(residual, "residual", x)
        if hidden is None:
            hidden, ldh = _rows_of_16_bytes(x, M, K, residual.dtype, stream)
        else:
            if hidden.dtype != residual.dtype:
                raise TypeError("hidden must have the residual's type")
            ldh = _rows_like(hidden, "hidden", x)
    elif hidden is not None:
        raise ValueError("hidden is written only with a residual")
    gp, gt = _gain(gain, K)
    y = q = scale = None
    yp = yt = ldy = qp = qt = ldq = sp = 0
    if out_dtype is not None:
        yt = _DTYPE_CODE.get(out_dtype)
        if yt is None:
            raise TypeError("out_dtype must be bf16, fp16, fp32 or None")
        y, ldy = _rows_of_16_bytes(x, M, K, out_dtype, stream)
        yp = y.data_ptr()
    if fp8_dtype is not None:
        qt = _FP8_CODE.get(fp8_dtype)
        if qt is None:
            raise TypeError("fp8_dtype must be torch.float8_e4m3fn, torch.float8_e5m2 or None")
        q, ldq = _rows_of_16_bytes(x, M, K, fp8_dtype, stream)
        scale = _empty(x, (_blocks(K), M), torch.float32, stream).t()
        qp, sp = q.data_ptr(), scale.data_ptr()
    elif y is None:
        raise ValueError("out_dtype and fp8_dtype are both None: nothing is wanted")
    row_scale = _empty(x, M, torch.float32, stream)
    _on_one_gpu("x residual hidden gain", x, residual, hidden, gain)
    status = load().tg_rmsnorm(
        _RMSNORM.pack(M, K, x.data_ptr(), ldx, _ptr(residual), ldr, gp, _ptr(hidden), ldh, yp, ldy, qp, ldq, sp, M,
                      row_scale.data_ptr(), eps, xt, rt, gt, yt, qt), _stream_handle(stream))
    if status:
        _check(status)
    return Normed(y, q, scale, x if hidden is None else hidden, row_scale)


def rmsnorm_backward(normed: Normed, dy: torch.Tensor, gain: torch.Tensor | None = None,
                     d_hidden: torch.Tensor | None = None, out: torch.Tensor | None = None, *,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(dx, d_gain): the gradients of rmsnorm's x (and residual: the same) and gain (tg_rmsnorm_backward).

    ``dy`` [M, K], bf16, fp16 or fp32, is the gradient of the normalised rows (the 8-bit copy counts as y itself),
    ``d_hidden`` (None: zero) what reaches ``normed.hidden`` past the norm, of its type.  ``out`` has hidden's type too
    and may be ``d_hidden``; ``d_gain`` is fp32 [K], None without a gain.
    """
    hidden, row_scale = normed.hidden, normed.row_scale
    ht, dt = _DTYPE_CODE.get(hidden.dtype), _DTYPE_CODE.get(dy.dtype)
    if ht is None or dt is None:
        raise TypeError("normed.hidden and dy must be bf16, fp16 or fp32")
    if hidden.dim() != 2:
        raise ValueError(f"normed.hidden must be 2-D, got shape {tuple(hidden.shape)}")
    M, K = hidden.shape
    ldh = _row_major_ld(hidden, "normed.hidden", K)
    lddy = _rows_like(dy, "dy", hidden)
    if row_scale.dtype != torch.float32 or row_scale.shape != (M,) or not row_scale.is_contiguous():
        raise ValueError(f"normed.row_scale must be a contiguous fp32 tensor {[M]}")
    gp, gt = _gain(gain, K)
    lddh = 0
    if d_hidden is not None:
        if d_hidden.dtype != hidden.dtype:
            raise TypeError("d_hidden must have hidden's type")
        lddh = _rows_like(d_hidden, "d_hidden", hidden)
    if out is None:
        out, ldo = _rows_of_16_bytes(hidden, M, K, hidden.dtype, stream)
    else:
        if out.dtype != hidden.dtype:
            raise TypeError("out must have hidden's type")
        ldo = _rows_like(out, "out", hidden)
    d_gain = None if gain is None else _empty(hidden, K, torch.float32, stream)
    _on_one_gpu("normed.hidden normed.row_scale dy gain d_hidden out", hidden, row_scale, dy, gain, d_hidden, out)
    status = load().tg_rmsnorm_backward(
        _RMSNORM_BACKWARD.pack(M, K, dy.data_ptr(), lddy, hidden.data_ptr(), ldh, row_scale.data_ptr(), gp,
                               _ptr(d_hidden), lddh, out.data_ptr(), ldo, _ptr(d_gain), dt, ht, gt),
        _stream_handle(stream))
    if status:
        _check(status)
    return out, d_gain


def lora_add(base: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapters: torch.Tensor,
             scale: torch.Tensor | None = None, out: torch.Tensor | None = None, *, stream=None) -> torch.Tensor:
    """out[t] = base[t] + scale[g] * (x[t] @ a[g].T) @ b[g].T with g = adapters[t]: each row's own low-rank adapter beside
    a shared projection (tg_lora_add).

    ``base`` [T, N] is the projection's result (gemm's or gemm_fp8's), bf16, fp16 or fp32; ``x`` [T, K], ``a`` [G, r, K] and
    ``b`` [G, N, r] are all bf16 or all fp16, their last dimension contiguous, r at most 128; ``adapters`` is an int32 CUDA
    tensor [T] in any order (rows of one request side by side are fastest), -1 (or any value outside [0, G)) for a row
    without; ``scale`` is fp32 [G].  ``out`` (allocated if not given) has base's shape and type and may be ``base``.
    Other rows never enter a row's result, but its last bits may be others in a batch of another size or with another
    number of adapters: the order of the sums goes by the sizes.
    """
    xt, bt = _DTYPE_CODE.get(x.dtype), _DTYPE_CODE.get(base.dtype)
    if xt is None or xt == F32 or a.dtype != x.dtype or b.dtype != x.dtype:
        raise TypeError("x, a and b must all be torch.bfloat16 or all torch.float16")
    if bt is None:
        raise TypeError("base must be bf16, fp16 or fp32")
    if base.dim() != 2 or x.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("shapes: base [T, N], x [T, K], a [G, r, K], b [G, N, r]")
    T, N = base.shape
    K = x.shape[1]
    G, r, _ = a.shape
    if x.shape[0] != T or a.shape[2] != K or b.shape != (G, N, r):
        raise ValueError(f"shapes: base [T, N], x [T, K], a [G, r, K], b [G, N, r]; got {list(base.shape)}, {list(x.shape)}, "
                         f"{list(a.shape)}, {list(b.shape)}")
    if adapters.dtype != torch.int32 or adapters.shape != (T,) or not adapters.is_contiguous():
        raise ValueError(f"adapters must be a contiguous int32 tensor {[T]}")
    if scale is not None and (scale.dtype != torch.float32 or scale.shape != (G,) or not scale.is_contiguous()):
        raise ValueError(f"scale must be a contiguous fp32 tensor {[G]}")
    ldx, ldbase = _row_major_ld(x, "x", K), _row_major_ld(base, "base", N)
    (sa, lda, a1), (sb, ldb, b1) = a.stride(), b.stride()
    if (a1 != 1 and K > 1) or (b1 != 1 and r > 1):
        raise ValueError("the last dimension of a and b must be contiguous")
    if out is None:
        out, ldo = _rows_of_16_bytes(base, T, N, base.dtype, stream)
    else:
        if out.dtype != base.dtype or out.shape != base.shape:
            raise ValueError("out must have base's shape and type")
        ldo = _row_major_ld(out, "out", N)
    _on_one_gpu("base x a b adapters scale out", base, x, a, b, adapters, scale, out)
    status = load().tg_lora_add(
        _LORA.pack(T, K, N, r, G, x.data_ptr(), ldx, a.data_ptr(), lda if r > 1 else K, sa if G > 1 else 0, b.data_ptr(),
                   ldb if N > 1 else r, sb if G > 1 else 0, adapters.data_ptr(), _ptr(scale), base.data_ptr(), ldbase,
                   out.data_ptr(), ldo, xt, bt), _stream_handle(stream))
    if status:
        _check(status)
    return out


class _Routing(NamedTuple):
    experts: torch.Tensor    # int32 [T, k], -1 where a row has no further expert
    weights: torch.Tensor    # fp32 [T, k]
    counts: torch.Tensor     # int32 [G]
    loss: torch.Tensor       # fp32, balance loss
    slope: torch.Tensor      # fp32 [G], d loss / d probability
    renormalize: bool


class Routing(_Routing):
    """What moe_router returns, and moe_router_backward needs again.

    A tuple of experts, weights, counts, loss, slope and renormalize.  With other scores, a bias, groups or a factor it has
    three more: ``score``, ``weight_scale`` and ``plain`` (false), so that one put together again from its entries does not
    lose them; the gate without those has the same three as attributes.
    """
    __slots__ = ()
    _fields = _Routing._fields + ("score", "weight_scale", "plain")

    def __new__(cls, experts, weights, counts, loss, slope, renormalize, score="softmax", weight_scale=1.0, plain=True):
        entries = (experts, weights, counts, loss, slope, renormalize)
        if not plain or score != "softmax" or weight_scale != 1.0:
            entries += (score, weight_scale, plain)
        return tuple.__new__(cls, entries)

    @property
    def score(self) -> str:
        return self[6] if len(self) > 6 else "softmax"

    @property
    def weight_scale(self) -> float:
        return self[7] if len(self) > 6 else 1.0

    @property
    def plain(self) -> bool:     # tg_moe_router's (softmax, no bias, groups or factor), whose gradient has a kernel of its own
        return len(self) == 6 or self[8]

    @classmethod
    def _make(cls, entries):
        return cls(*entries)

    def _replace(self, **fields):
        return type(self)(**{**self._asdict(), **fields})

    def __repr__(self) -> str:
        return f"Routing({', '.join(f'{k}={v!r}' for k, v in self._asdict().items())})"


def _logits(logits: torch.Tensor) -> tuple[int, int, int, int]:
    """(type code, T, G, ld) of a row-major [T, G] matrix of logits."""
    dt = _DTYPE_CODE.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be bf16, fp16 or fp32")
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D, got shape {tuple(logits.shape)}")
    T, G = logits.shape
    return dt, T, G, _row_major_ld(logits, "logits", G)


def moe_router(logits: torch.Tensor, top_k: int, *, renormalize: bool = False, score: str = "softmax",
               bias: torch.Tensor | None = None, groups: int = 1, top_groups: int | None = None, group_top: int = 1,
               weight_scale: float = 1.0, stream=None) -> Routing:
    """Top-k experts of each token, their weights, per-expert counts and balance loss (tg_moe_router, tg_moe_router_scored).

    ``logits`` is row-major [T, G] bf16, fp16 or fp32; -infinity forbids an expert, a row of it is padding.
    ``counts`` is what moe_gemm_device and moe_gemm_fp8 read; the loss is G * sum(f * P), 1 when all is even.

    ``score`` is "softmax" or "sigmoid".  ``bias`` (fp32 [G]) is added to the scores for the choice alone, not for the
    weights.  With ``groups`` groups of neighbouring experts, only the ``top_groups`` best are chosen from (None: all),
    a group's score being the sum of its ``group_top`` (1 or 2) largest.  The weights are times ``weight_scale``.
    """
    dt, T, G, ld = _logits(logits)
    if not isinstance(top_k, int) or top_k < 1:
        raise ValueError("top_k must be a positive integer")
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (G,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous fp32 tensor {[G]}")
    _on_one_gpu("logits bias", logits, bias)
    shape = (T, top_k)
    plain = (code == 0 and bias is None and groups == 1 and weight_scale == 1.0 and top_groups in (None, 1) and group_top == 1)
    r = Routing(_empty(logits, shape, torch.int32, stream), _empty(logits, shape, torch.float32, stream),
                _empty(logits, G, torch.int32, stream), _empty(logits, (), torch.float32, stream),
                _empty(logits, G, torch.float32, stream), bool(renormalize), score, float(weight_scale), plain)
    if plain:
        status = load().tg_moe_router(logits.data_ptr(), dt, ld, T, G, top_k, int(renormalize), r.experts.data_ptr(),
                                      r.weights.data_ptr(), r.counts.data_ptr(), r.loss.data_ptr(), r.slope.data_ptr(),
                                      _stream_handle(stream))
    else:
        status = load().tg_moe_router_scored(
            _ROUTER.pack(T, G, top_k, logits.data_ptr(), ld, _ptr(bias), groups, groups if top_groups is None else top_groups,
                         group_top, r.experts.data_ptr(), r.weights.data_ptr(), r.counts.data_ptr(), r.loss.data_ptr(),
                         r.slope.data_ptr(), r.weight_scale, dt, code, r.renormalize), _stream_handle(stream))
    if status:
        _check(status)
    return r


def moe_router_backward(logits: torch.Tensor, routing: Routing, d_weights: torch.Tensor | None = None,
                        d_loss: torch.Tensor | None = None, out: torch.Tensor | None = None, *,
                        stream=None) -> torch.Tensor:
    """The gradient of ``logits`` from those of routing.weights (fp32 [T, k]) and routing.loss (fp32, one
    element, on the GPU); None is zero (tg_moe_router_backward).  ``out`` has the logits' type."""
    dt, T, G, ld = _logits(logits)
    code = SCORES.get(routing.score)
    if code is None:
        raise ValueError(f"routing.score must be one of {sorted(SCORES)}, got {routing.score!r}")
    k = routing.experts.shape[1]
    experts, weights, slope = routing.experts, routing.weights, routing.slope
    if experts.dtype != torch.int32 or experts.shape[0] != T or not experts.is_contiguous():
        raise ValueError(f"routing.experts must be a contiguous int32 tensor {[T, k]}")
    if weights.dtype != torch.float32 or weights.shape != experts.shape or not weights.is_contiguous():
        raise ValueError(f"routing.weights must be a contiguous fp32 tensor {[T, k]}")
    if slope.dtype != torch.float32 or tuple(slope.shape) != (G,) or not slope.is_contiguous():
        raise ValueError(f"routing.slope must be a contiguous fp32 tensor {[G]}")
    if d_weights is not None and (d_weights.dtype != torch.float32 or d_weights.shape != experts.shape
                                  or not d_weights.is_contiguous()):
        raise ValueError(f"d_weights must be a contiguous fp32 tensor {[T, k]}")
    if d_loss is not None and (d_loss.dtype != torch.float32 or d_loss.numel() != 1):
        raise ValueError("d_loss must be an fp32 tensor of one element")
    if out is None:
        out, ldd = _empty(logits, (T, G), logits.dtype, stream), max(G, 1)
    else:
        if out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out must be [T, G] of the logits' type")
        ldd = _row_major_ld(out, "out", G)
    _on_one_gpu("logits routing.experts routing.weights routing.slope d_weights d_loss out", logits, experts,
                weights, slope, d_weights, d_loss, out)
    if routing.plain and code == 0 and routing.weight_scale == 1.0:
        status = load().tg_moe_router_backward(logits.data_ptr(), dt, ld, T, G, k, int(routing.renormalize),
                                               experts.data_ptr(), weights.data_ptr(), slope.data_ptr(),
                                               None if d_weights is None else d_weights.data_ptr(),
                                               None if d_loss is None else d_loss.data_ptr(), out.data_ptr(), ldd,
                                               _stream_handle(stream))
    else:
        status = load().tg_moe_router_scored_backward(
            _ROUTER_BACKWARD.pack(T, G, k, logits.data_ptr(), ld, experts.data_ptr(), slope.data_ptr(), _ptr(d_weights),
                                  _ptr(d_loss), out.data_ptr(), ldd, routing.weight_scale, dt,
                                  code, routing.renormalize), _stream_handle(stream))
    if status:
        _check(status)
    return out


def make_problem(a, b, out, *, bias=None, epilogue="none") -> GroupProblem:
    """One tg_group_problem from tensors (a may have 0 rows: an empty group)."""
    M, K = a.shape
    _, N = b.shape
    la, lda = _matrix(a, "a") if a.numel() else (ROW_MAJOR, max(K, 1))
    lb, ldb = _matrix(b, "b")
    _, ldc = _matrix(out, "out") if out.numel() else (ROW_MAJOR, max(N, 1))
    epi = EPILOGUES[epilogue]
    return GroupProblem(M, N, K, _ptr(a) if a.numel() else None, lda, la, _ptr(b), ldb, lb,
                        _ptr(out) if out.numel() else None, ldc, _DTYPE_CODE[out.dtype], epi,
                        _ptr(bias) if epi else None, F16 if b.dtype == torch.float16 else BF16)


def grouped_gemm_table(table, stream=None) -> None:
    """Call tg_grouped_gemm on a sequence of GroupProblem (or a ctypes array of them)."""
    arr = table if isinstance(table, ctypes.Array) else (GroupProblem * len(table))(*table)
    _check(load().tg_grouped_gemm(arr, len(arr), _stream_handle(stream)))


def grouped_gemm_table_noalloc(table, stream=None) -> None:
    """tg_grouped_gemm_noalloc: the same grouped GEMM with its problem table in the
    library's fixed device array (no device allocation; at most 256 non-empty problems)."""
    arr = table if isinstance(table, ctypes.Array) else (GroupProblem * len(table))(*table)
    _check(load().tg_grouped_gemm_noalloc(arr, len(arr), _stream_handle(stream)))


def build_moe_table(a: torch.Tensor, b: torch.Tensor, counts, out: torch.Tensor, *, bias: torch.Tensor | None = None,
                    epilogue: str = "none") -> ctypes.Array:
    """The tg_group_problem table of an MoE expert GEMM (see moe_grouped_gemm), built once for reuse."""
    counts = [int(c) for c in counts]
    G = len(counts)
    if b.dim() != 3 or b.shape[0] != G:
        raise ValueError("b must be [G, K, N] with G = len(counts)")
    total = sum(counts)
    if a.shape[0] != total or out.shape[0] != total:
        raise ValueError(f"a and out need {total} rows (sum of counts)")
    table = []
    r = 0
    for g, m in enumerate(counts):
        table.append(make_problem(a[r:r + m], b[g], out[r:r + m], bias=None if bias is None else bias[g],
                                  epilogue=epilogue))
        r += m
    return (GroupProblem * G)(*table)


def moe_grouped_gemm(a: torch.Tensor, b: torch.Tensor, counts, out: torch.Tensor | None = None, *,
                     bias: torch.Tensor | None = None, epilogue: str = "none",
                     out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """MoE expert GEMM: rows of ``a`` [sum M_g, K] grouped by expert (``counts`` on the host),
    expert g's rows times ``b[g]`` ([G, K, N], each a row- or column-major view) into ``out`` [sum M_g, N].
    ``bias`` is [G, N] bf16 when the epilogue uses one."""
    if out is None:
        out = torch.empty((a.shape[0], b.shape[2]), dtype=out_dtype, device=a.device)
    grouped_gemm_table(build_moe_table(a, b, counts, out, bias=bias, epilogue=epilogue), stream)
    return out


def device_status(stream=None) -> None:
    """Synchronise ``stream`` and raise TGError if a kernel reported a timeout or CUDA failed."""
    _check(load().tg_device_status(_stream_handle(stream)))


def set_wait_budget_ms(ms: int) -> None:
    _check(load().tg_set_wait_budget_ms(ms))


def debug_withhold_stage(k_block: int, block: int = 0) -> None:
    """Arm the failure-path test hook for this thread's next launch (tg_debug_withhold_stage_in)."""
    _check(load().tg_debug_withhold_stage_in(k_block, block))


def debug_trace(tile_records: torch.Tensor | None, cta_records: torch.Tensor | None = None) -> None:
    """Arm a timeline trace of this thread's next launch (see tg_debug_trace in include/tg.h).

    ``tile_records`` is an int64 CUDA tensor [T, 4] and ``cta_records`` [B, 4]; the
    capacities passed to the library are T and B records of four stamps each."""
    for name, t in (("tile_records", tile_records), ("cta_records", cta_records)):
        if t is not None and (t.dim() != 2 or t.shape[1] != 4 or t.dtype != torch.int64 or not t.is_contiguous()
                              or not t.is_cuda):
            raise ValueError(f"{name} must be a contiguous int64 CUDA tensor of shape [n, 4]")
    tp = 0 if tile_records is None else tile_records.data_ptr()
    tc = 0 if tile_records is None else tile_records.shape[0]
    cp = 0 if cta_records is None else cta_records.data_ptr()
    cc = 0 if cta_records is None else cta_records.shape[0]
    _check(load().tg_debug_trace(tp or None, tc, cp or None, cc))


def launch_count() -> int:
    """Kernels this thread has enqueued through libtg so far (tg_launch_count)."""
    return int(load().tg_launch_count())


def version() -> tuple[int, int]:
    v = load().tg_version()
    return v >> 16, v & 0xFFFF
