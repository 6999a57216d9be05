"""Python binding of libfp8moe.so (the C ABI in include/fp8moe.h).

Argument marshalling only: it checks dtypes/devices/contiguity, allocates the
outputs (and, when the caller passes none, the workspace) with torch, and passes
raw device pointers, sizes and the current CUDA stream to the library. Every
step of the computation runs in the library's CUDA kernels; if the library is
missing or fails to load, every call raises.

Function names follow the C ABI without the ``fp8moe_`` prefix.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import threading
from typing import Optional

import torch

from . import build as _build

OK = 0
ERRORS = {-1: "EINVAL", -2: "EALIGN", -3: "EWORKSPACE", -4: "ECUDA", -5: "EUNSUPPORTED"}

OP_GMM_FP8_FWD = 1
OP_GMM_SILU_FP8_FWD = 2
OP_GMM_DLHS_FP8 = 3
OP_TGMM_DRHS_QUANT = 4
OP_GMM_BF16_FWD = 5
OP_GMM_FP8_FWD_BLOCK = 7
OP_GMM_MXFP4_FWD = 8
OP_GMM_SILU_MXFP4_FWD = 9
OP_NORM_BWD = 10
OP_BALANCE = 11

STATUS_NEGATIVE_GROUP = 0x1
STATUS_GROUPS_EXCEED_M = 0x2
STATUS_WAIT_TIMEOUT = 0x4
STATUS_BAD_EXPERT = 0x10
STATUS_BAD_OFFSETS = 0x20

# every symbol include/fp8moe.h declares
EXPORTS = [
    "fp8moe_workspace_size", "fp8moe_gmm_fp8_fwd", "fp8moe_gmm_silu_fp8_fwd",
    "fp8moe_gmm_dlhs_fp8", "fp8moe_gmm_dlhs_fp8_path", "fp8moe_tgmm_drhs_quant",
    "fp8moe_dequantize_fp8_codes", "fp8moe_gmm_bf16_fwd", "fp8moe_quantize_rows",
    "fp8moe_tgmm_quantize_tiles", "fp8moe_read_status", "fp8moe_status_string",
    "fp8moe_last_cuda_error", "fp8moe_num_sms", "fp8moe_gmm_silu_fp8_fwd_noalloc",
    "fp8moe_gmm_dlhs_dswiglu_fp8", "fp8moe_gmm_dlhs_dswiglu_fp8_path",
    "fp8moe_tgmm_drhs_quant_fmt", "fp8moe_tgmm_quantize_tiles_fmt",
    "fp8moe_gmm_fp8_fwd_block", "fp8moe_quantize_rows_block", "fp8moe_selftest_wait_timeout",
    "fp8moe_selftest_cast_f32", "fp8moe_sort_tokens", "fp8moe_dispatch_tokens",
    "fp8moe_combine_tokens", "fp8moe_combine_tokens_bwd", "fp8moe_norm_fwd", "fp8moe_norm_bwd",
    "fp8moe_mxfp4_quantize_rows", "fp8moe_mxfp4_quantize_weights", "fp8moe_mxfp4_dequantize",
    "fp8moe_gmm_mxfp4_fwd", "fp8moe_gmm_silu_mxfp4_fwd",
    "fp8moe_router_fwd", "fp8moe_balance_fwd", "fp8moe_router_bwd", "fp8moe_adamw_workspace_size",
    "fp8moe_adamw_step",
]

FMT = {"e4m3": 0, "e5m2": 1}

_lock = threading.Lock()
_lib = None


class Fp8MoeError(RuntimeError):
    pass


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load (building first if needed) the shared library and declare the ABI."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise Fp8MoeError(f"libfp8moe.so not built ({path})")
            _build.build()
        L = ctypes.CDLL(path)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        F32, F64, U32 = ctypes.c_float, ctypes.c_double, ctypes.c_uint32
        sig = {
            "fp8moe_workspace_size": ([I32, I64, I64, I64, I32], SZ),
            "fp8moe_gmm_fp8_fwd": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, P], I32),
            "fp8moe_gmm_silu_fp8_fwd": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, P], I32),
            "fp8moe_gmm_dlhs_fp8": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, P], I32),
            "fp8moe_gmm_dlhs_fp8_path": ([P, I64, I64, P, P, I32, I64, P, P, I32, P], I32),
            "fp8moe_tgmm_drhs_quant": ([P, P, I64, I64, I64, I32, P, P, P, SZ, P], I32),
            "fp8moe_dequantize_fp8_codes": ([P, P, I32, I64, I64, P, P], I32),
            "fp8moe_gmm_bf16_fwd": ([P, I64, I64, P, I32, I64, P, I32, P, P], I32),
            "fp8moe_quantize_rows": ([P, I64, I64, P, I32, P, P, P], I32),
            "fp8moe_tgmm_quantize_tiles": ([P, P, I64, I64, I64, I32, P, P, P, P, P, P], I32),
            "fp8moe_read_status": ([P, ctypes.POINTER(ctypes.c_uint32)], I32),
            "fp8moe_status_string": ([I32], ctypes.c_char_p),
            "fp8moe_last_cuda_error": ([], I32),
            "fp8moe_num_sms": ([], I32),
            "fp8moe_gmm_silu_fp8_fwd_noalloc": ([P, I64, I64, P, P, I32, I64, P, P, P], I32),
            "fp8moe_gmm_dlhs_dswiglu_fp8": ([P, I64, I64, P, P, I32, I64, P, P, P, P, SZ, P], I32),
            "fp8moe_gmm_dlhs_dswiglu_fp8_path": ([P, I64, I64, P, P, I32, I64, P, P, P, I32, P],
                                                 I32),
            "fp8moe_tgmm_drhs_quant_fmt": ([P, P, I64, I64, I64, I32, P, P, P, SZ, I32, P], I32),
            "fp8moe_tgmm_quantize_tiles_fmt": ([P, P, I64, I64, I64, I32, P, P, P, P, P, I32, P],
                                               I32),
            "fp8moe_gmm_fp8_fwd_block": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, I32, I32, P],
                                         I32),
            "fp8moe_quantize_rows_block": ([P, I64, I64, P, I32, I32, P, P, P], I32),
            "fp8moe_selftest_wait_timeout": ([ctypes.c_uint32, P], I32),
            "fp8moe_selftest_cast_f32": ([P, I64, I32, P, P], I32),
            "fp8moe_sort_tokens": ([P, I64, I32, I32, I64, P, P, P, P], I32),
            "fp8moe_dispatch_tokens": ([P, P, I64, I32, I64, I32, I32, I64, P, P, P, P, P], I32),
            "fp8moe_combine_tokens": ([P, I64, I64, I32, P, P, I64, I32, P, P], I32),
            "fp8moe_combine_tokens_bwd": ([P, P, I64, I64, I32, P, P, I64, I32, P, P, P], I32),
            "fp8moe_norm_fwd": ([P, P, I64, I64, I32, P, P, P, I32, I32, F32, F32, F32, P, P, P, P,
                                 P], I32),
            "fp8moe_norm_bwd": ([P, P, P, P, I64, I64, I32, P, P, P, P, P, I32, I32, F32, F32, P, P,
                                 P, P, P, P, SZ, P], I32),
            "fp8moe_mxfp4_quantize_rows": ([P, I64, I64, P, I32, P, P, P], I32),
            "fp8moe_mxfp4_quantize_weights": ([P, I32, I64, I64, P, P, P], I32),
            "fp8moe_mxfp4_dequantize": ([P, P, I32, I64, I64, P, P], I32),
            "fp8moe_gmm_mxfp4_fwd": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, P], I32),
            "fp8moe_gmm_silu_mxfp4_fwd": ([P, I64, I64, P, P, I32, I64, P, P, P, SZ, P], I32),
            "fp8moe_router_fwd": ([P, I64, I32, I32, I32, P, I32, I32, F32, P, I32, P, P, P, P, P, P,
                                   SZ, P], I32),
            "fp8moe_balance_fwd": ([P, P, I64, I32, I32, I32, I32, P, I32, P, P, P, P, SZ, P], I32),
            "fp8moe_router_bwd": ([P, P, P, I64, I32, I32, I32, I32, I32, F32, P, P, P, I32, P, P],
                                  I32),
            "fp8moe_adamw_workspace_size": ([P, I32, I32], SZ),
            "fp8moe_adamw_step": ([P, I32, I64, P, F64, P, F64, F64, F64, P, U32, P, SZ, P], I32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
        return _lib


def _check(rc: int, what: str):
    if rc != OK:
        L = load()
        msg = L.fp8moe_status_string(rc).decode()
        extra = ""
        if rc == -4:
            extra = f" (cudaError {L.fp8moe_last_cuda_error()})"
        raise Fp8MoeError(f"{what}: {ERRORS.get(rc, rc)} -- {msg}{extra}")


def _ptr(t: Optional[torch.Tensor]):
    return t.data_ptr() if t is not None else None


# the stream's handle without a Stream object around it, where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _req(t: torch.Tensor, dtype, name: str, ndim: int):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.dim() == ndim \
            and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@functools.lru_cache(maxsize=1024)
def workspace_size(op: int, M: int, K: int, N: int, E: int) -> int:
    return int(load().fp8moe_workspace_size(op, M, K, N, E))


def _workspace(op, M, K, N, E, device, workspace):
    need = workspace_size(op, M, K, N, E)
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


def _fwd(lhs, codes, scale, group_sizes, out, workspace, silu: bool):
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    E, K2, N = codes.shape
    if K2 != K or scale.shape != (E, N) or group_sizes.numel() != E:
        raise ValueError("shape mismatch")
    Nout = N // 2 if silu else N
    if out is None:
        out = torch.empty(M, Nout, dtype=torch.bfloat16, device=lhs.device)
    else:
        _req(out, torch.bfloat16, "out", 2)
        if out.shape != (M, Nout):
            raise ValueError("out shape")
    op = OP_GMM_SILU_FP8_FWD if silu else OP_GMM_FP8_FWD
    ws, wsb = _workspace(op, M, K, N, E, lhs.device, workspace)
    fn = L.fp8moe_gmm_silu_fp8_fwd if silu else L.fp8moe_gmm_fp8_fwd
    _check(fn(_ptr(lhs), M, K, _ptr(codes), _ptr(scale), E, N, _ptr(group_sizes), _ptr(out),
              _ptr(ws), wsb, _stream(lhs.device)), fn.__name__)
    return out


def gmm_fp8_fwd(lhs, codes, scale, group_sizes, out=None, workspace=None):
    """wo forward: bf16 [M, N] (see fp8moe_gmm_fp8_fwd)."""
    return _fwd(lhs, codes, scale, group_sizes, out, workspace, silu=False)


def gmm_silu_fp8_fwd(lhs, codes, scale, group_sizes, out=None, workspace=None):
    """wi forward with fused SwiGLU: bf16 [M, N/2] (see fp8moe_gmm_silu_fp8_fwd)."""
    return _fwd(lhs, codes, scale, group_sizes, out, workspace, silu=True)


def gmm_fp8_fwd_block(lhs, codes, scale, group_sizes, swiglu: bool, out=None, workspace=None,
                      block: int = 512):
    """Forward GMM with per-512-column block activation scales and bf16
    accumulation across blocks (see fp8moe_gmm_fp8_fwd_block)."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    E, K2, N = codes.shape
    if K2 != K or scale.shape != (E, N) or group_sizes.numel() != E:
        raise ValueError("shape mismatch")
    Nout = N // 2 if swiglu else N
    if out is None:
        out = torch.empty(M, Nout, dtype=torch.bfloat16, device=lhs.device)
    else:
        _req(out, torch.bfloat16, "out", 2)
    ws, wsb = _workspace(OP_GMM_FP8_FWD_BLOCK, M, K, N, E, lhs.device, workspace)
    _check(L.fp8moe_gmm_fp8_fwd_block(_ptr(lhs), M, K, _ptr(codes), _ptr(scale), E, N,
                                      _ptr(group_sizes), _ptr(out), _ptr(ws), wsb, block,
                                      1 if swiglu else 0, _stream(lhs.device)),
           "fp8moe_gmm_fp8_fwd_block")
    return out


def quantize_rows_block(lhs, group_sizes, block: int = 512):
    """Parity export of the per-block activation quantization: codes u8 [M, K]
    and bf16-valued f32 scales [M, ceil(K / block)]."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    nb = (K + block - 1) // block
    q = torch.zeros(M, K, dtype=torch.uint8, device=lhs.device)
    sb = torch.full((M, nb), float("nan"), dtype=torch.float32, device=lhs.device)
    _check(L.fp8moe_quantize_rows_block(_ptr(lhs), M, K, _ptr(group_sizes), group_sizes.numel(),
                                        block, _ptr(q), _ptr(sb), _stream(lhs.device)),
           "fp8moe_quantize_rows_block")
    return q, sb


NOALLOC_SCRATCH_BYTES = 32 << 20


def gmm_silu_fp8_fwd_noalloc(lhs, codes, scale, group_sizes, out):
    """wi forward without a caller workspace: the library's fixed 32 MiB device
    array stands in for it (see fp8moe_gmm_silu_fp8_fwd_noalloc). ``out`` must be
    given; this call allocates nothing."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    _req(out, torch.bfloat16, "out", 2)
    M, K = lhs.shape
    E, _, N = codes.shape
    _check(L.fp8moe_gmm_silu_fp8_fwd_noalloc(_ptr(lhs), M, K, _ptr(codes), _ptr(scale), E, N,
                                             _ptr(group_sizes), _ptr(out), _stream(lhs.device)),
           "fp8moe_gmm_silu_fp8_fwd_noalloc")
    return out


def gmm_dlhs_fp8(dout, codes, scale, group_sizes, out=None, path: Optional[int] = None):
    """dLHS: bf16 [M, K] (see fp8moe_gmm_dlhs_fp8; path forces 0 streaming /
    1 cached / 2 CTA pairs with the weight in tensor memory)."""
    L = load()
    _req(dout, torch.bfloat16, "dout", 2)
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, N = dout.shape
    E, K, N2 = codes.shape
    if N2 != N or scale.shape != (E, N) or group_sizes.numel() != E:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty(M, K, dtype=torch.bfloat16, device=dout.device)
    else:
        _req(out, torch.bfloat16, "out", 2)
    st = _stream(dout.device)
    if path is None:
        rc = L.fp8moe_gmm_dlhs_fp8(_ptr(dout), M, N, _ptr(codes), _ptr(scale), E, K,
                                   _ptr(group_sizes), _ptr(out), None, 0, st)
    else:
        rc = L.fp8moe_gmm_dlhs_fp8_path(_ptr(dout), M, N, _ptr(codes), _ptr(scale), E, K,
                                        _ptr(group_sizes), _ptr(out), int(path), st)
    _check(rc, "fp8moe_gmm_dlhs_fp8")
    return out


def gmm_dlhs_dswiglu_fp8(dout, codes, scale, gu, group_sizes, out=None,
                         path: Optional[int] = None):
    """wo dLHS + SwiGLU backward: dgu bf16 [M, 2F] from dout [M, N], the wo
    codes [E, F, N] and the wi output gu [M, 2F] (see fp8moe_gmm_dlhs_dswiglu_fp8;
    path forces 0 streaming / 1 cached / 2 CTA pairs)."""
    L = load()
    _req(dout, torch.bfloat16, "dout", 2)
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    _req(gu, torch.bfloat16, "gu", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, N = dout.shape
    E, F, N2 = codes.shape
    if N2 != N or scale.shape != (E, N) or group_sizes.numel() != E or gu.shape != (M, 2 * F):
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=dout.device)
    else:
        _req(out, torch.bfloat16, "out", 2)
    st = _stream(dout.device)
    if path is None:
        rc = L.fp8moe_gmm_dlhs_dswiglu_fp8(_ptr(dout), M, N, _ptr(codes), _ptr(scale), E, F,
                                           _ptr(gu), _ptr(group_sizes), _ptr(out), None, 0, st)
    else:
        rc = L.fp8moe_gmm_dlhs_dswiglu_fp8_path(_ptr(dout), M, N, _ptr(codes), _ptr(scale), E,
                                                F, _ptr(gu), _ptr(group_sizes), _ptr(out),
                                                int(path), st)
    _check(rc, "fp8moe_gmm_dlhs_dswiglu_fp8")
    return out


def tgmm_drhs_quant(lhs, dout, group_sizes, out=None, workspace=None, dout_fmt: str = "e4m3"):
    """Weight gradient f32 [E, K, N] (see fp8moe_tgmm_drhs_quant; dout_fmt
    "e5m2" quantizes the gradient operand to e5m2, fp8moe_tgmm_drhs_quant_fmt)."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(dout, torch.bfloat16, "dout", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    M2, N = dout.shape
    if M2 != M:
        raise ValueError("shape mismatch")
    E = group_sizes.numel()
    if out is None:
        out = torch.empty(E, K, N, dtype=torch.float32, device=lhs.device)
    else:
        _req(out, torch.float32, "out", 3)
    ws, wsb = _workspace(OP_TGMM_DRHS_QUANT, M, K, N, E, lhs.device, workspace)
    if dout_fmt == "e4m3":
        rc = L.fp8moe_tgmm_drhs_quant(_ptr(lhs), _ptr(dout), M, K, N, E, _ptr(group_sizes),
                                      _ptr(out), _ptr(ws), wsb, _stream(lhs.device))
    else:
        rc = L.fp8moe_tgmm_drhs_quant_fmt(_ptr(lhs), _ptr(dout), M, K, N, E, _ptr(group_sizes),
                                          _ptr(out), _ptr(ws), wsb, FMT[dout_fmt],
                                          _stream(lhs.device))
    _check(rc, "fp8moe_tgmm_drhs_quant")
    return out


def dequantize_fp8_codes(codes, scale, out=None):
    """bf16 [E, K, N] = bf16(code * scale) (see fp8moe_dequantize_fp8_codes)."""
    L = load()
    _req(codes, torch.uint8, "codes", 3)
    _req(scale, torch.float32, "scale", 2)
    E, K, N = codes.shape
    if out is None:
        out = torch.empty(E, K, N, dtype=torch.bfloat16, device=codes.device)
    _check(L.fp8moe_dequantize_fp8_codes(_ptr(codes), _ptr(scale), E, K, N, _ptr(out),
                                         _stream(codes.device)), "fp8moe_dequantize_fp8_codes")
    return out


def gmm_bf16_fwd(lhs, w, group_sizes, swiglu: bool, out=None):
    """BF16 comparison GMM (see fp8moe_gmm_bf16_fwd)."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(w, torch.bfloat16, "w", 3)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    E, K2, N = w.shape
    if K2 != K:
        raise ValueError("shape mismatch")
    Nout = N // 2 if swiglu else N
    if out is None:
        out = torch.empty(M, Nout, dtype=torch.bfloat16, device=lhs.device)
    _check(L.fp8moe_gmm_bf16_fwd(_ptr(lhs), M, K, _ptr(w), E, N, _ptr(group_sizes),
                                 int(bool(swiglu)), _ptr(out), _stream(lhs.device)),
           "fp8moe_gmm_bf16_fwd")
    return out


def quantize_rows(lhs, group_sizes, q=None, sx=None):
    """Parity export: codes u8 [M, K] and scales f32 [M] for rows < T."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    if q is None:
        q = torch.zeros(M, K, dtype=torch.uint8, device=lhs.device)
    if sx is None:
        sx = torch.full((M,), float("nan"), dtype=torch.float32, device=lhs.device)
    _check(L.fp8moe_quantize_rows(_ptr(lhs), M, K, _ptr(group_sizes), group_sizes.numel(),
                                  _ptr(q), _ptr(sx), _stream(lhs.device)), "fp8moe_quantize_rows")
    return q, sx


def segment_bound(M: int, E: int) -> int:
    return (M + 127) // 128 + E


def tgmm_quantize_tiles(lhs, dout, group_sizes, dout_fmt: str = "e4m3"):
    """Parity export of the tgmm operand quantization (slot layout)."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(dout, torch.bfloat16, "dout", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    _, N = dout.shape
    E = group_sizes.numel()
    S = segment_bound(M, E)
    dev = lhs.device
    qx = torch.zeros(S, 128, K, dtype=torch.uint8, device=dev)
    sx = torch.full((S, K), float("nan"), dtype=torch.float32, device=dev)
    qd = torch.zeros(S, 128, N, dtype=torch.uint8, device=dev)
    sd = torch.full((S, N), float("nan"), dtype=torch.float32, device=dev)
    _check(L.fp8moe_tgmm_quantize_tiles_fmt(_ptr(lhs), _ptr(dout), M, K, N, E, _ptr(group_sizes),
                                            _ptr(qx), _ptr(sx), _ptr(qd), _ptr(sd), FMT[dout_fmt],
                                            _stream(dev)),
           "fp8moe_tgmm_quantize_tiles")
    return qx, sx, qd, sd


def selftest_wait_timeout(limit_us: int, device=None) -> None:
    """Enqueue the bounded-wait failure self-test (see fp8moe_selftest_wait_timeout)."""
    _check(load().fp8moe_selftest_wait_timeout(int(limit_us), _stream(device)),
           "fp8moe_selftest_wait_timeout")


def selftest_cast_f32(x, fmt: str = "e4m3", codes=None):
    """The quantizers' f32 -> fp8 cast on arbitrary f32 values (a device tensor):
    codes u8 of x's shape (see fp8moe_selftest_cast_f32)."""
    _req(x, torch.float32, "x", x.dim())
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(load().fp8moe_selftest_cast_f32(_ptr(x), x.numel(), FMT[fmt], _ptr(codes),
                                           _stream(x.device)), "fp8moe_selftest_cast_f32")
    return codes


TYPES = {torch.bfloat16: 0, torch.float32: 1}
GATES = {"token": 1, "channel": 2, "full": 3}


def _req_rows(t: torch.Tensor, name: str) -> int:
    """Checks a contiguous [rows, H] CUDA tensor of a row type; the type's number."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    ty = TYPES.get(t.dtype)
    if ty is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    _req(t, t.dtype, name, 2)
    return ty


def _shaped(t, dtype, name: str, shape: tuple):
    """_req with the whole shape."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.shape == shape \
            and t.is_contiguous():
        return
    _req(t, dtype, name, len(shape))
    raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _like(out, shape, dtype, device, name: str):
    """A given output, checked, or a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _shaped(out, dtype, name, shape)
    return out


def _sort_outputs(ids, num_experts: int, M: int):
    T, k = ids.shape
    i32, dev = torch.int32, ids.device
    return (torch.empty(num_experts, dtype=i32, device=dev),
            torch.empty(T, k, dtype=i32, device=dev), torch.empty(M, dtype=i32, device=dev))


def sort_tokens(ids, num_experts: int, M: Optional[int] = None):
    """The router's choices ids int32 [T, topk] sorted by expert: (group_sizes [E],
    slot_row [T, topk], row_slot [M]), all int32 (see fp8moe_sort_tokens). M: rows
    of the sorted buffer, T * topk by default."""
    L = load()
    _req(ids, torch.int32, "ids", 2)
    T, k = ids.shape
    M = T * k if M is None else int(M)
    gs, slot_row, row_slot = _sort_outputs(ids, num_experts, M)
    _check(L.fp8moe_sort_tokens(_ptr(ids), T, k, num_experts, M, _ptr(gs), _ptr(slot_row),
                                _ptr(row_slot), _stream(ids.device)), "fp8moe_sort_tokens")
    return gs, slot_row, row_slot


def dispatch_tokens(x, ids, num_experts: int, M: Optional[int] = None, out=None):
    """x [T, H] (bf16 or f32) copied to its tokens' rows, sorted by expert:
    (rows [M, H], group_sizes, slot_row, row_slot) (see fp8moe_dispatch_tokens).
    Rows past the last group's are not written."""
    L = load()
    ty = _req_rows(x, "x")
    _req(ids, torch.int32, "ids", 2)
    T, H = x.shape
    if ids.shape[0] != T:
        raise ValueError("shape mismatch")
    k = ids.shape[1]
    M = T * k if M is None else int(M)
    out = _like(out, (M, H), x.dtype, x.device, "out")
    gs, slot_row, row_slot = _sort_outputs(ids, num_experts, M)
    _check(L.fp8moe_dispatch_tokens(_ptr(x), _ptr(ids), T, k, H, ty, num_experts, M, _ptr(out),
                                    _ptr(gs), _ptr(slot_row), _ptr(row_slot), _stream(x.device)),
           "fp8moe_dispatch_tokens")
    return out, gs, slot_row, row_slot


def combine_tokens(rows, slot_row, weights=None, out=None):
    """out [T, H] = sum_j weights[t, j] * rows[slot_row[t, j]] in f32, weights f32
    [T, topk] or None for ones (see fp8moe_combine_tokens)."""
    L = load()
    ty = _req_rows(rows, "rows")
    _req(slot_row, torch.int32, "slot_row", 2)
    M, H = rows.shape
    T, k = slot_row.shape
    if weights is not None:
        _shaped(weights, torch.float32, "weights", (T, k))
    out = _like(out, (T, H), rows.dtype, rows.device, "out")
    _check(L.fp8moe_combine_tokens(_ptr(rows), M, H, ty, _ptr(slot_row), _ptr(weights), T, k,
                                   _ptr(out), _stream(rows.device)), "fp8moe_combine_tokens")
    return out


def dispatch_tokens_bwd(drows, slot_row, out=None):
    """Gradient of dispatch_tokens with respect to x [T, H]: the sum of a token's
    rows' gradients."""
    return combine_tokens(drows, slot_row, None, out)


def combine_tokens_bwd(dout, rows, slot_row, weights, out=None):
    """Gradient of combine_tokens: (drows [M, H], dweights f32 [T, topk]) (see
    fp8moe_combine_tokens_bwd). Rows of drows that no slot names are not written."""
    L = load()
    ty = _req_rows(rows, "rows")
    _req(slot_row, torch.int32, "slot_row", 2)
    M, H = rows.shape
    T, k = slot_row.shape
    _shaped(dout, rows.dtype, "dout", (T, H))
    _shaped(weights, torch.float32, "weights", (T, k))
    out = _like(out, (M, H), rows.dtype, rows.device, "out")
    dweights = torch.empty(T, k, dtype=torch.float32, device=rows.device)
    _check(L.fp8moe_combine_tokens_bwd(_ptr(dout), _ptr(rows), M, H, ty, _ptr(slot_row),
                                       _ptr(weights), T, k, _ptr(out), _ptr(dweights),
                                       _stream(rows.device)), "fp8moe_combine_tokens_bwd")
    return out, dweights


def _gate(gate, kind: Optional[str], T: int, H: int, dtype):
    """The gate's kind number and the shape and type that it (and its gradient) has."""
    if (gate is None) != (kind is None):
        raise ValueError("gate and gate_kind go together")
    if gate is None:
        return 0, None, None
    if kind not in GATES:
        raise ValueError(f"gate_kind must be one of {sorted(GATES)}, got {kind!r}")
    shape = (T,) if kind == "token" else (H,) if kind == "channel" else (T, H)
    ty = dtype if kind == "full" else torch.float32
    _shaped(gate, ty, f"a gate per {kind}", shape)
    return GATES[kind], shape, ty


def norm_fwd(x, y=None, w_post=None, w_pre=None, gate=None, gate_kind: Optional[str] = None,
             sigmoid: bool = False, residual_scale: float = 1.0, branch_scale: float = 1.0,
             eps: float = 1e-6):
    """The norms after and before a block with its gate and the scaled residual sum:
        r = residual_scale * x + branch_scale * g * (w_post * rmsnorm(y))
        h = w_pre * rmsnorm(r)
    Returns (r, h, rstd_post, rstd_pre); without y and w_post r is x and returned as
    None (the scales belong to the sum and are not used), without w_pre h and rstd_pre
    are None. gate_kind: "token" (f32 [T]),
    "channel" (f32 [H]) or "full" ([T, H] of x's type); sigmoid passes the gate
    through one (see fp8moe_norm_fwd)."""
    L = load()
    ty = _req_rows(x, "x")
    T, H = x.shape
    post, pre = w_post is not None, w_pre is not None
    if (y is not None) != post:
        raise ValueError("y and w_post go together")
    if not post and gate is not None:
        raise ValueError("a gate needs y and w_post")
    f32, dev = torch.float32, x.device
    kind = _gate(gate, gate_kind, T, H, x.dtype)[0] if gate is not None or gate_kind is not None else 0
    r = h = rstd_post = rstd_pre = None
    if post:
        _shaped(y, x.dtype, "y", (T, H))
        _shaped(w_post, f32, "w_post", (H,))
        r = torch.empty_like(x)
        rstd_post = torch.empty(T, dtype=f32, device=dev)
    if pre:
        _shaped(w_pre, f32, "w_pre", (H,))
        h = torch.empty_like(x)
        rstd_pre = torch.empty(T, dtype=f32, device=dev)
    _check(L.fp8moe_norm_fwd(_ptr(x), _ptr(y), T, H, ty, _ptr(w_post), _ptr(w_pre), _ptr(gate),
                             kind, int(bool(sigmoid)), residual_scale, branch_scale, eps, _ptr(r),
                             _ptr(h), _ptr(rstd_post), _ptr(rstd_pre), _stream(dev)),
           "fp8moe_norm_fwd")
    return r, h, rstd_post, rstd_pre


def norm_bwd(dr, dh, r, y=None, w_post=None, w_pre=None, rstd_post=None, rstd_pre=None, gate=None,
             gate_kind: Optional[str] = None, sigmoid: bool = False, residual_scale: float = 1.0,
             branch_scale: float = 1.0, workspace=None):
    """Gradient of norm_fwd: (dx, dy, dw_post, dw_pre, dgate), None for what the
    forward did not have. dr: the residual stream's gradient of r (None: zero); dh:
    of h; r: the forward's r, or its x when it had no y (see fp8moe_norm_bwd)."""
    L = load()
    like = dr if dr is not None else dh
    if like is None:
        raise ValueError("dr or dh must be given")
    ty = _req_rows(like, "dr" if dr is not None else "dh")
    T, H = like.shape
    dt, dev, f32 = like.dtype, like.device, torch.float32
    post, pre = w_post is not None, w_pre is not None
    if (y is not None) != post or (rstd_post is not None) != post:
        raise ValueError("y, w_post and rstd_post go together")
    if (dh is not None) != pre or (rstd_pre is not None) != pre or (pre and r is None):
        raise ValueError("dh, w_pre, rstd_pre and r go together")
    if not post and gate is not None:
        raise ValueError("a gate needs y and w_post")
    rows = (T, H)
    if dh is not None and like is not dh:
        _shaped(dh, dt, "dh", rows)
    if pre:
        _shaped(r, dt, "r", rows)
        _shaped(w_pre, f32, "w_pre", (H,))
        _shaped(rstd_pre, f32, "rstd_pre", (T,))
    if post:
        _shaped(y, dt, "y", rows)
        _shaped(w_post, f32, "w_post", (H,))
        _shaped(rstd_post, f32, "rstd_post", (T,))
    kind, gshape, gtype = _gate(gate, gate_kind, T, H, dt)
    dx = torch.empty(T, H, dtype=dt, device=dev)
    dy = torch.empty(T, H, dtype=dt, device=dev) if post else None
    dw_post = torch.empty(H, dtype=f32, device=dev) if post else None
    dw_pre = torch.empty(H, dtype=f32, device=dev) if pre else None
    dgate = torch.empty(gshape, dtype=gtype, device=dev) if kind else None
    ws, wsb = _workspace(OP_NORM_BWD, T, H, 0, 0, dev, workspace)
    _check(L.fp8moe_norm_bwd(_ptr(dr), _ptr(dh), _ptr(r) if pre else None, _ptr(y), T, H, ty,
                             _ptr(w_post), _ptr(w_pre), _ptr(rstd_post), _ptr(rstd_pre),
                             _ptr(gate), kind, int(bool(sigmoid)), residual_scale, branch_scale,
                             _ptr(dx), _ptr(dy), _ptr(dw_post), _ptr(dw_pre), _ptr(dgate), _ptr(ws),
                             wsb, _stream(dev)), "fp8moe_norm_bwd")
    return dx, dy, dw_post, dw_pre, dgate


def mxfp4_words(K: int) -> int:
    """32-bit scale words of a row: one for every 128 values along K."""
    return (K + 127) // 128


def mxfp4_quantize_rows(lhs, group_sizes):
    """Parity export of the 4-bit products' activation quantization: codes u8
    [M, K/2] and scales u8 [ceil(K/128), M, 4] for rows < T (others zero)."""
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    M, K = lhs.shape
    codes = torch.zeros(M, K // 2, dtype=torch.uint8, device=lhs.device)
    scales = torch.zeros(mxfp4_words(K), M, 4, dtype=torch.uint8, device=lhs.device)
    _check(L.fp8moe_mxfp4_quantize_rows(_ptr(lhs), M, K, _ptr(group_sizes), group_sizes.numel(),
                                        _ptr(codes), _ptr(scales), _stream(lhs.device)),
           "fp8moe_mxfp4_quantize_rows")
    return codes, scales


def mxfp4_quantize_weights(w):
    """Expert weights bf16 [E, K, N] as MXFP4 with blocks along K: codes u8
    [E, N, K/2] and scales u8 [E, ceil(K/128), N, 4] (see
    fp8moe_mxfp4_quantize_weights)."""
    L = load()
    _req(w, torch.bfloat16, "w", 3)
    E, K, N = w.shape
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(E, mxfp4_words(K), N, 4, dtype=torch.uint8, device=w.device)
    _check(L.fp8moe_mxfp4_quantize_weights(_ptr(w), E, K, N, _ptr(codes), _ptr(scales),
                                           _stream(w.device)), "fp8moe_mxfp4_quantize_weights")
    return codes, scales


def _mxfp4_weight(codes, scales):
    _req(codes, torch.uint8, "codes", 3)
    E, N, half = codes.shape
    K = 2 * half
    _shaped(scales, torch.uint8, "scales", (E, mxfp4_words(K), N, 4))
    return E, K, N


def mxfp4_dequantize(codes, scales, out=None):
    """bf16 [E, N, K] of MXFP4 weights: K contiguous, so that as the weight of
    gmm_bf16_fwd it gives a product's activation gradient (see
    fp8moe_mxfp4_dequantize)."""
    L = load()
    E, K, N = _mxfp4_weight(codes, scales)
    out = _like(out, (E, N, K), torch.bfloat16, codes.device, "out")
    _check(L.fp8moe_mxfp4_dequantize(_ptr(codes), _ptr(scales), E, N, K, _ptr(out),
                                     _stream(codes.device)), "fp8moe_mxfp4_dequantize")
    return out


def _mxfp4_fwd(lhs, codes, scales, group_sizes, out, workspace, silu: bool):
    L = load()
    _req(lhs, torch.bfloat16, "lhs", 2)
    _req(group_sizes, torch.int32, "group_sizes", 1)
    E, K, N = _mxfp4_weight(codes, scales)
    M, K2 = lhs.shape
    if K2 != K or group_sizes.numel() != E:
        raise ValueError("shape mismatch")
    out = _like(out, (M, N // 2 if silu else N), torch.bfloat16, lhs.device, "out")
    op = OP_GMM_SILU_MXFP4_FWD if silu else OP_GMM_MXFP4_FWD
    ws, wsb = _workspace(op, M, K, N, E, lhs.device, workspace)
    fn = L.fp8moe_gmm_silu_mxfp4_fwd if silu else L.fp8moe_gmm_mxfp4_fwd
    _check(fn(_ptr(lhs), M, K, _ptr(codes), _ptr(scales), E, N, _ptr(group_sizes), _ptr(out),
              _ptr(ws), wsb, _stream(lhs.device)), fn.__name__)
    return out


def gmm_mxfp4_fwd(lhs, codes, scales, group_sizes, out=None, workspace=None):
    """Grouped product of 4-bit weights with the rows quantised to 4 bits: bf16
    [M, N] (see fp8moe_gmm_mxfp4_fwd)."""
    return _mxfp4_fwd(lhs, codes, scales, group_sizes, out, workspace, silu=False)


def gmm_silu_mxfp4_fwd(lhs, codes, scales, group_sizes, out=None, workspace=None):
    """The same with fused SwiGLU: bf16 [M, N/2] (see fp8moe_gmm_silu_mxfp4_fwd)."""
    return _mxfp4_fwd(lhs, codes, scales, group_sizes, out, workspace, silu=True)


SCORES = {"softmax": 0, "sigmoid": 1}


def _router(logits, score: str, topk: int, seq_offsets):
    """Checks what the router's calls share: (type number, score number, B)."""
    ty = TYPES.get(logits.dtype) if isinstance(logits, torch.Tensor) else None
    if ty is None or not logits.is_cuda or logits.dim() != 2 or not logits.is_contiguous():
        ty = _req_rows(logits, "logits")
    sc = SCORES.get(score)
    if sc is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    B = 1
    if seq_offsets is not None:
        _req(seq_offsets, torch.int32, "seq_offsets", 1)
        B = seq_offsets.numel() - 1
        if B < 1:
            raise ValueError("seq_offsets must hold at least one sequence (two offsets)")
    return ty, sc, B


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _one_device(device, *tensors) -> None:
    """Every tensor of a call (or None) lies on the current device."""
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors must be on {device}, got one on {t.device}")
    if index != _current_device():
        raise ValueError(f"tensors must be on the current device, got {device}")


def _balance_outputs(B: int, E: int, device):
    return (torch.empty(B, E, dtype=torch.int32, device=device),
            torch.empty(B, dtype=torch.float32, device=device),
            torch.empty(B, E, dtype=torch.float32, device=device))


def router_fwd(logits, topk: int, score: str = "softmax", bias=None, normalize: bool = True,
               weight_scale: float = 1.0, balance: bool = False, seq_offsets=None, workspace=None):
    """The router's choice for logits [T, E] (bf16 or f32): (ids int32 [T, topk], weights f32
    [T, topk], counts, loss, slope), the last three None unless balance (see
    fp8moe_router_fwd and balance_fwd). score: "softmax" or "sigmoid"; bias f32 [E] takes part in
    the choice alone; normalize: a token's weights add up to weight_scale. seq_offsets int32
    [B + 1]: where the sequences of the batch begin and end; tokens outside get no expert (-1)."""
    L = load()
    ty, sc, B = _router(logits, score, topk, seq_offsets)
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        _shaped(bias, torch.float32, "bias", (E,))
    _one_device(dev, bias, seq_offsets, workspace)
    if topk < 1:
        raise ValueError("topk must be positive")
    ids = torch.empty(T, topk, dtype=torch.int32, device=dev)
    weights = torch.empty(T, topk, dtype=torch.float32, device=dev)
    counts = loss = slope = None
    ws, wsb = None, 0
    if balance:
        counts, loss, slope = _balance_outputs(B, E, dev)
        ws, wsb = _workspace(OP_BALANCE, T, 0, B, E, dev, workspace)
    rc = L.fp8moe_router_fwd(logits.data_ptr(), T, E, ty, sc, _ptr(bias), topk, 1 if normalize else 0,
                             weight_scale, _ptr(seq_offsets), B, ids.data_ptr(), weights.data_ptr(),
                             _ptr(counts), _ptr(loss), _ptr(slope), _ptr(ws), wsb, _stream(dev))
    if rc:
        _check(rc, "fp8moe_router_fwd")
    return ids, weights, counts, loss, slope


def balance_fwd(logits, ids, score: str = "softmax", seq_offsets=None, workspace=None):
    """The balance loss of given choices ids int32 [T, topk]: (counts int32 [B, E], loss f32 [B],
    slope f32 [B, E]) for each sequence (see fp8moe_balance_fwd): loss = sum_i slope_i * sum of the
    tokens' shares of expert i, slope_i = E counts_i / (choices * tokens). router_fwd gives the
    same in its pass over the logits."""
    L = load()
    _req(ids, torch.int32, "ids", 2)
    T, k = ids.shape
    ty, sc, B = _router(logits, score, k, seq_offsets)
    if logits.shape[0] != T:
        raise ValueError("shape mismatch")
    E, dev = logits.shape[1], logits.device
    _one_device(dev, ids, seq_offsets, workspace)
    counts, loss, slope = _balance_outputs(B, E, dev)
    ws, wsb = _workspace(OP_BALANCE, T, 0, B, E, dev, workspace)
    _check(L.fp8moe_balance_fwd(_ptr(logits), _ptr(ids), T, E, ty, sc, k, _ptr(seq_offsets), B,
                                _ptr(counts), _ptr(loss), _ptr(slope), _ptr(ws), wsb, _stream(dev)),
           "fp8moe_balance_fwd")
    return counts, loss, slope


def router_bwd(dweights, logits, ids, score: str = "softmax", normalize: bool = True,
               weight_scale: float = 1.0, dloss=None, slope=None, seq_offsets=None, out=None):
    """Gradient into the logits [T, E], of their type: of the weights (dweights f32 [T, topk], or
    None) and of the balance losses (dloss f32 [B] with the forward's slope, or None) (see
    fp8moe_router_bwd). ids and the options: the forward's."""
    L = load()
    _req(ids, torch.int32, "ids", 2)
    T, k = ids.shape
    ty, sc, B = _router(logits, score, k, seq_offsets)
    if logits.shape[0] != T:
        raise ValueError("shape mismatch")
    E, dev, f32 = logits.shape[1], logits.device, torch.float32
    if (dloss is None) != (slope is None):
        raise ValueError("dloss and slope go together")
    if dweights is not None:
        _shaped(dweights, f32, "dweights", (T, k))
    if dloss is not None:
        _shaped(dloss, f32, "dloss", (B,))
        _shaped(slope, f32, "slope", (B, E))
    _one_device(dev, ids, dweights, dloss, slope, seq_offsets, out)
    out = _like(out, (T, E), logits.dtype, dev, "out")
    _check(L.fp8moe_router_bwd(_ptr(dweights), _ptr(logits), _ptr(ids), T, E, ty, sc, k,
                               int(bool(normalize)), weight_scale, _ptr(dloss), _ptr(slope),
                               _ptr(seq_offsets), B, _ptr(out), _stream(dev)), "fp8moe_router_bwd")
    return out


class _AdamwTensor(ctypes.Structure):
    """fp8moe_adamw_tensor."""
    _fields_ = ([(n, ctypes.c_uint64) for n in ("p", "g", "m", "v", "m_scale", "v_scale", "copy",
                                                "codes", "code_scale")] +
                [(n, ctypes.c_int64) for n in ("n", "K", "N")] +
                [("weight_decay", ctypes.c_double), ("g_type", ctypes.c_int32),
                 ("state_bits", ctypes.c_int32)])


# whether tensors lie at their addresses still, in one call where torch has one (900 tensors: 30 us,
# 53 otherwise)
_addresses_equal = getattr(
    torch._C, "_tensors_data_ptrs_at_indices_equal",
    lambda tensors, at, places: list(map(torch.Tensor.data_ptr, tensors)) == at)

ADAMW_BLOCK = 128  # consecutive values of an 8-bit moment that share a scale


def adamw_blocks(n: int) -> int:
    """Scales of an 8-bit moment of n values."""
    return -(-n // ADAMW_BLOCK)


class AdamwPlan:
    """The tensors of adamw_step, checked once: f32 params with their moments, in 32 bits (f32
    of the same shape) or, where m_scales and v_scales are given, in 8 (u8 codes of the same
    shape, f32 [ceil(n / 128)] scales; zeros to begin with). copies: bf16 copies of the new
    params; codes and code_scales: u8 [E, K, N] and f32 [E, N], the 8-bit weights of params
    [E, K, N]. Each is a list as long as params, with None where a param has none, or None.
    weight_decay: a number or one for each param. The plan keeps the tensors' memory: where one of
    them has other memory than it had (its data replaced, or grown), adamw_step refuses the plan;
    a new one takes 4 to 8 us a param."""

    def __init__(self, params, m, v, m_scales=None, v_scales=None, copies=None, codes=None,
                 code_scales=None, weight_decay=0.0):
        count = len(params)
        none = [None] * count

        def listed(x, name):
            if x is None:
                return none
            if len(x) != count:
                raise ValueError(f"{name} must have one entry for each of the {count} params")
            return list(x)

        m, v = listed(m, "m"), listed(v, "v")
        m_scales, v_scales = listed(m_scales, "m_scales"), listed(v_scales, "v_scales")
        copies, codes = listed(copies, "copies"), listed(codes, "codes")
        code_scales = listed(code_scales, "code_scales")
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) \
            else [float(weight_decay)] * count
        listed(decay, "weight_decay")
        self.params, self._kept, self._shapes = list(params), [], []
        self._tensors, self._addresses, self._names = [], [], []
        self.device = None
        self._table = (_AdamwTensor * max(1, count))()
        f32, u8, bf16 = torch.float32, torch.uint8, torch.bfloat16
        spans, index = [], None

        def enter(e, i, t, field, dtype, shape, name):
            """Checks a tensor and writes its address down; its memory is kept."""
            nonlocal index
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                    and t.is_cuda and t.is_contiguous()):
                _shaped(t, dtype, f"{name} {i}", tuple(shape))
            if t.get_device() != index:
                if index is not None:
                    raise ValueError(f"param {i} and its states must be on {self.device}")
                self.device, index = t.device, t.get_device()
            at = t.data_ptr()
            setattr(e, field, at)
            spans.append((at, at + t.nbytes, i))
            self._kept.append(t.untyped_storage())
            self._tensors.append(t)
            self._addresses.append(at)
            self._names.append((name, i))

        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor):
                raise TypeError(f"param {i} must be a tensor")
            shape, n, e = p.shape, p.numel(), self._table[i]
            enter(e, i, p, "p", f32, shape, "param")
            eight = m_scales[i] is not None
            if eight != (v_scales[i] is not None):
                raise ValueError(f"m_scale and v_scale of param {i} go together")
            state = u8 if eight else f32
            enter(e, i, m[i], "m", state, shape, "m of param")
            enter(e, i, v[i], "v", state, shape, "v of param")
            if eight:
                blocks = (adamw_blocks(n),)
                enter(e, i, m_scales[i], "m_scale", f32, blocks, "m_scale of param")
                enter(e, i, v_scales[i], "v_scale", f32, blocks, "v_scale of param")
            if copies[i] is not None:
                enter(e, i, copies[i], "copy", bf16, shape, "copy of param")
            if (codes[i] is None) != (code_scales[i] is None):
                raise ValueError(f"codes and code_scale of param {i} go together")
            if codes[i] is not None:
                if len(shape) != 3:
                    raise ValueError(f"param {i} must be [E, K, N] to have codes, got {tuple(shape)}")
                enter(e, i, codes[i], "codes", u8, shape, "codes of param")
                enter(e, i, code_scales[i], "code_scale", f32, (shape[0], shape[2]),
                      "code_scale of param")
                e.K, e.N = shape[1], shape[2]
            e.n, e.weight_decay, e.state_bits = n, float(decay[i]), 8 if eight else 32
            self._shapes.append(shape)
        spans = sorted(s for s in spans if s[0] < s[1])
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError(f"params {a[2]} and {b[2]} or their states overlap")
        self._places = list(range(len(self._tensors)))
        self._indices = [index] * count
        self._numels = array.array("Q", [p.numel() for p in self.params])
        self._columns = memoryview(self._table).cast("B").cast("Q") if count else None
        # what a backward pass may have kept, and autograd is told of: weights and what is made of
        # them, by the tensors whose version counters they share, one for a tensor's views
        self._made = [[t if (base := t._base) is None else base for t in ts if t is not None]
                      for ts in zip(self.params, copies, codes, code_scales)]
        made = {id(t): t for ts in self._made for t in ts}
        if any(map(torch.Tensor.is_inference, made.values())):      # these have no counters
            self._made = [[t for t in ts if not t.is_inference()] for ts in self._made]
            made = {id(t): t for ts in self._made for t in ts}
        self._all_made = list(made.values())
        self._type = None                       # of all gradients in the table
        self._lock = threading.Lock()           # the table is one call's until the library read it

    def _enter(self, grads):
        """Writes the gradients' addresses and types into the table; returns it, its length, and
        the tensors whose versions the step raises."""
        count = len(self.params)
        if len(grads) != count:
            raise ValueError(f"grads must have one entry for each of the {count} params")
        if not _addresses_equal(self._tensors, self._addresses, self._places):
            for t, at, (name, i) in zip(self._tensors, self._addresses, self._names):
                if t.data_ptr() != at:
                    raise ValueError(f"the storage of {name} {i} was replaced: make a new plan")
        table, dev = self._table, self.device
        try:                                    # the usual case, column by column
            types = [g.dtype for g in grads]
            if types.count(types[0]) == count and types[0] in TYPES \
                    and [g.shape for g in grads] == self._shapes \
                    and all(map(torch.Tensor.is_contiguous, grads)) \
                    and list(map(torch.Tensor.get_device, grads)) == self._indices:
                words, step = self._columns, ctypes.sizeof(_AdamwTensor) // 8
                words[_AdamwTensor.g.offset // 8::step] = \
                    array.array("Q", map(torch.Tensor.data_ptr, grads))
                words[_AdamwTensor.n.offset // 8::step] = self._numels
                if self._type != types[0]:
                    for e in table[:count]:
                        e.g_type = TYPES[types[0]]
                    self._type = types[0]
                return table, count, self._all_made
        except (AttributeError, TypeError):     # something is no tensor
            pass
        self._type = None
        made = {}
        for i, g in enumerate(grads):
            e = table[i]
            if g is None:                       # no gradient: the param is left as it is
                e.n = 0
                continue
            ty = TYPES.get(g.dtype) if isinstance(g, torch.Tensor) else None
            if ty is None or g.shape != self._shapes[i] or g.device != dev \
                    or not g.is_contiguous():
                if not isinstance(g, torch.Tensor):
                    raise TypeError(f"gradient {i} must be a tensor")
                if ty is None:
                    raise TypeError(f"gradient {i} must be torch.bfloat16 or torch.float32, got "
                                    f"{g.dtype}")
                _shaped(g, g.dtype, f"gradient {i}", tuple(self._shapes[i]))
                raise ValueError(f"gradient {i} must be on {dev}, got {g.device}")
            e.g, e.g_type, e.n = g.data_ptr(), ty, g.numel()
            made.update((id(t), t) for t in self._made[i])
        return table, count, list(made.values())


def adamw_step(plan: AdamwPlan, grads, step, lr, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, grad_scale=None, seed: int = 0, workspace=None) -> None:
    """One AdamW step on the plan's tensors, in place, for grads (bf16 or f32, one for each param;
    None leaves the param and its states as they are) (see fp8moe_adamw_step). step: the number
    of this step, from 1, or an int64 CUDA tensor [1]; lr: a number or an f32 CUDA tensor [1] (what
    a captured step reads when it is replayed). grad_scale: f32 CUDA tensor [1] that every gradient
    is multiplied by, or None. seed: of the rounding of 8-bit moments. Autograd sees params, copies
    and codes as changed in place."""
    L = load()
    if not plan.params:
        return
    dev = plan.device
    step_dev = lr_dev = None
    if isinstance(step, torch.Tensor):
        _shaped(step, torch.int64, "step", (1,))
        step, step_dev = 0, step
    if isinstance(lr, torch.Tensor):
        _shaped(lr, torch.float32, "lr", (1,))
        lr, lr_dev = 0.0, lr
    if grad_scale is not None:
        _shaped(grad_scale, torch.float32, "grad_scale", (1,))
    _one_device(dev, step_dev, lr_dev, grad_scale, workspace)
    if workspace is not None and not (workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    with plan._lock:
        table, count, made = plan._enter(grads)
        need = int(L.fp8moe_adamw_workspace_size(table, count,
                                                 step_dev is not None or lr_dev is not None))
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(L.fp8moe_adamw_step(table, count, int(step), _ptr(step_dev), float(lr),
                                   _ptr(lr_dev), beta1, beta2, eps, _ptr(grad_scale),
                                   seed & 0xFFFFFFFF, _ptr(workspace), wsb, _stream(dev)),
               "fp8moe_adamw_step")
        torch.autograd.graph.increment_version(made)


def read_status(device=None) -> int:
    """Synchronize the current stream and return (and clear) the status bits."""
    L = load()
    flags = ctypes.c_uint32(0)
    _check(L.fp8moe_read_status(_stream(device), ctypes.byref(flags)), "fp8moe_read_status")
    return int(flags.value)


def num_sms() -> int:
    return int(load().fp8moe_num_sms())
