"""Python binding of libdg, the GB300 (sm_103a) fine-grained-scaled FP8 GEMM library.

Argument marshalling only: every function below passes device pointers, sizes and the
current CUDA stream to the C ABI declared in include/dg.h; all arithmetic runs in the
library's CUDA kernels. There is no fallback: if libdg.so is missing or the call
fails, an exception is raised.

The GEMM computes D = C + A @ B.T (DeepGEMM README, "Interfaces / Notices", as
reproduced on the page "Weight gradient kernels for dense and MoE models #95"), with
A and B in E4M3, UE8M0 scales packed four per int32 (A: per row per 128-K group,
B: per 128x128 block), FP32 accumulation and a BF16 result.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK = 0
STATUS_NAMES = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED", 3: "DG_ERR_MISALIGNED",
                4: "DG_ERR_CUDA", 5: "DG_ERR_TIMEOUT", 6: "DG_ERR_BAD_INDEX"}

# (name, restype, argtypes) of every entry point in include/dg.h
_P = ctypes.c_void_p
_I = ctypes.c_int
SIGNATURES = [
    ("dg_fp8_gemm_nt", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_wgrad_gemm_fp8_fp8_fp32_nt", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_fp8_gemm_nn", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_fp8_gemm_tn", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_fp8_gemm_tt", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_k_grouped_wgrad_gemm_fp8_fp8_fp32_nt", _I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    ("dg_k_grouped_fp8_gemm_tn_contiguous", _I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    ("dg_m_grouped_fp8_gemm_nn_contiguous", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_m_grouped_fp8_gemm_nt_contiguous", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_m_grouped_fp8_gemm_nt_masked", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_fp8_fp4_gemm_nt", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_m_grouped_fp8_fp4_gemm_nt_contiguous", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_m_grouped_fp8_fp4_gemm_nt_masked", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_pack_sf_ue8m0", _I, [_P, _P, _I, _I, _I, _P]),
    ("dg_add_rms_norm", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    ("dg_add_rms_norm_backward", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_moe_route", _I, [_P, _P, _P, _P, _P]),
    ("dg_moe_route_backward", _I, [_P, _P, _P, _P, _P, _P]),
    ("dg_moe_fp8_few_tokens", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    ("dg_moe_fp8_fp4_few_tokens", _I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    ("dg_get_mk_alignment_for_contiguous_layout", _I, []),
    ("dg_set_mk_alignment_for_contiguous_layout", _I, [_I]),
    ("dg_get_theoretical_mk_alignment_for_contiguous_layout", _I, []),
    ("dg_get_tma_aligned_size", _I, [_I, _I]),
    ("dg_set_num_sms", _I, [_I]),
    ("dg_reserve_workspace", _I, [_P, ctypes.c_size_t]),
    ("dg_release_workspace", _I, [_P]),
    ("dg_get_workspace_size", ctypes.c_size_t, [_P]),
    ("dg_set_pdl", _I, [_I]),
    ("dg_get_pdl", _I, []),
    ("dg_get_num_sms", _I, []),
    ("dg_get_device_status", _I, [_P]),
    ("dg_status_string", ctypes.c_char_p, [_I]),
    ("dg_last_cuda_error", _I, []),
    ("dg_set_debug", _I, [_I, ctypes.c_ulonglong]),
    ("dg_measure_fp8_mma_tflops", _I, [_I, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
    ("dg_quantize_fp4", _I, [_P, _P, _P, _P, _P, _P]),
    ("dg_swiglu_quantize_fp4", _I, [_P, _P, _P, _P, _P, _P]),
    ("dg_swiglu_backward", _I, [_P, _P, _P, _P, _P, _P]),
    ("dg_moe_balance_loss", _I, [_P, _P, _P, _P, _P, _P, _P, _P]),
    ("dg_moe_balance_loss_backward", _I, [_P, _P, _P, _P, _P, _P, _P, _P]),
    ("dg_fp4_gemm_nt", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    ("dg_m_grouped_fp4_gemm_nt_contiguous", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_m_grouped_fp4_gemm_nt_masked", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    ("dg_fp8_gemm_nt_no_alloc", _I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
]


class DGError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libdg.so (built by fp8_gemm_nt_gb300.build) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m fp8_gemm_nt_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    # the raw handle: torch.cuda.current_stream() would build a Stream object for every call (3 us)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(name: str, status: int) -> None:
    if status != DG_OK:
        raise DGError(name, status)


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _here(t: torch.Tensor, name: str) -> None:
    # the library works on the current device (and its stream): memory of another GPU would be
    # read through the wrong device's mappings
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _fp8(t: torch.Tensor, name: str) -> None:
    _here(t, name)
    _need(t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
    _need(t.dtype in (torch.float8_e4m3fn, torch.uint8), f"{name} must be float8_e4m3fn (or its uint8 bytes)")


def _i32(t: torch.Tensor, name: str) -> None:
    _here(t, name)
    _need(t.is_contiguous() and t.dtype == torch.int32, f"{name} must be a contiguous CUDA int32 tensor")


def _bf16(t: torch.Tensor, name: str) -> None:
    _here(t, name)
    _need(t.is_contiguous() and t.dtype == torch.bfloat16, f"{name} must be a contiguous CUDA bf16 tensor")


def _f32(t: torch.Tensor, name: str) -> None:
    _here(t, name)
    _need(t.is_contiguous() and t.dtype == torch.float32, f"{name} must be a contiguous CUDA float32 tensor")


def sf_shape(mn: int, k: int, groups: Optional[int] = None):
    """Shape of a packed scale tensor for an MN extent and K: [(G,) ceil(K/512), ceil4(mn)]."""
    shape = (-(-(k // 128) // 4), 4 * (-(-mn // 4)))
    return shape if groups is None else (groups,) + shape


def dg_fp8_gemm_nt(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A @ B.T. a [M, K] e4m3, sfa [KP, ceil4(M)] int32, b [N, K] e4m3,
    sfb [KP, ceil4(ceil(N/128))] int32, c [M, N] bf16 or None, d [M, N] bf16 (written)."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d")
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K and tuple(d.shape) == (M, N), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K), "scale shape mismatch")
    if c is not None:
        _bf16(c, "c")
        _need(tuple(c.shape) == (M, N), "c shape mismatch")
    _check("dg_fp8_gemm_nt", lib.dg_fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                                M, N, K, _stream(stream)))
    return d


def _dense_layout(name, a_kmajor, b_kmajor, a, sfa, b, sfb, c, d, stream):
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d")
    M, K = a.shape if a_kmajor else a.shape[::-1]
    N = b.shape[0] if b_kmajor else b.shape[1]
    Kb = b.shape[1] if b_kmajor else b.shape[0]
    _need(Kb == K and tuple(d.shape) == (M, N), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K), "scale shape mismatch")
    if c is not None:
        _bf16(c, "c")
        _need(tuple(c.shape) == (M, N), "c shape mismatch")
    _check(name, getattr(lib, name)(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d), M, N, K,
                                    _stream(stream)))
    return d


def dg_fp8_gemm_nn(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A @ B with a [M, K] (K-major) and b [K, N] (N-major); scales as dg_fp8_gemm_nt."""
    return _dense_layout("dg_fp8_gemm_nn", True, False, a, sfa, b, sfb, c, d, stream)


def dg_fp8_gemm_tn(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A.T @ B with a [K, M] (M-major, M a multiple of 16) and b [K, N]."""
    return _dense_layout("dg_fp8_gemm_tn", False, False, a, sfa, b, sfb, c, d, stream)


def dg_fp8_gemm_tt(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A.T @ B.T with a [K, M] (M-major, M a multiple of 16) and b [N, K]."""
    return _dense_layout("dg_fp8_gemm_tt", False, True, a, sfa, b, sfb, c, d, stream)


def dg_wgrad_gemm_fp8_fp8_fp32_nt(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """Weight-gradient GEMM, D = C + A @ B.T with FP32 C and D (C may be D itself, which then
    accumulates in place). a, sfa, b, sfb as dg_fp8_gemm_nt; c [M, N] float32 or None;
    d [M, N] float32 (written)."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _f32(d, "d")
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K and tuple(d.shape) == (M, N), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K), "scale shape mismatch")
    if c is not None:
        _f32(c, "c")
        _need(tuple(c.shape) == (M, N), "c shape mismatch")
    _check("dg_wgrad_gemm_fp8_fp8_fp32_nt",
           lib.dg_wgrad_gemm_fp8_fp8_fp32_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                             M, N, K, _stream(stream)))
    return d


def dg_k_grouped_wgrad_gemm_fp8_fp8_fp32_nt(a, sfa, b, sfb, c, d, ks, stream=None) -> torch.Tensor:
    """K-grouped weight-gradient GEMM: D[g] = C[g] + A[:, slice_g] @ B[:, slice_g].T in FP32,
    expert g owning the K-slice of length ks[g]. a [M, K_total] e4m3, sfa [R, ceil4(M)] int32
    (packed per expert, R word rows), b [N, K_total], sfb [R, ceil4(ceil(N/128))],
    c [G, M, N] float32 or None (may be d), d [G, M, N] float32, ks [G] int32 (CUDA)."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _f32(d, "d"); _i32(ks, "ks")
    M, K = a.shape
    N = b.shape[0]
    G = ks.shape[0]
    _need(b.shape[1] == K and tuple(d.shape) == (G, M, N), "shape mismatch")
    R = sfa.shape[0]
    _need(sfa.dim() == 2 and sfa.shape[1] == 4 * (-(-M // 4)) and sfb.dim() == 2 and sfb.shape[0] == R
          and sfb.shape[1] == 4 * (-(-(-(-N // 128)) // 4)), "scale shape mismatch")
    if c is not None:
        _f32(c, "c")
        _need(tuple(c.shape) == (G, M, N), "c shape mismatch")
    _check("dg_k_grouped_wgrad_gemm_fp8_fp8_fp32_nt",
           lib.dg_k_grouped_wgrad_gemm_fp8_fp8_fp32_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                                       _ptr(ks), G, M, N, K, R, _stream(stream)))
    return d


def dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, c, d, ks, stream=None) -> torch.Tensor:
    """K-grouped GEMM, TN layout: a [K_total, M] e4m3 (M a multiple of 16), b [K_total, N] e4m3,
    scales packed per expert as for dg_k_grouped_wgrad_gemm_fp8_fp8_fp32_nt, c [G, M, N] float32
    or None (may be d), d [G, M, N] float32, ks [G] int32 (CUDA)."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _f32(d, "d"); _i32(ks, "ks")
    K, M = a.shape
    Kb, N = b.shape
    G = ks.shape[0]
    _need(Kb == K and tuple(d.shape) == (G, M, N), "shape mismatch")
    R = sfa.shape[0]
    _need(sfa.dim() == 2 and sfa.shape[1] == 4 * (-(-M // 4)) and sfb.dim() == 2 and sfb.shape[0] == R
          and sfb.shape[1] == 4 * (-(-(-(-N // 128)) // 4)), "scale shape mismatch")
    if c is not None:
        _f32(c, "c")
        _need(tuple(c.shape) == (G, M, N), "c shape mismatch")
    _check("dg_k_grouped_fp8_gemm_tn_contiguous",
           lib.dg_k_grouped_fp8_gemm_tn_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                                   _ptr(ks), G, M, N, K, R, _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nn_contiguous(a, sfa, b, sfb, d, m_indices, stream=None) -> torch.Tensor:
    """Contiguous M-grouped GEMM with N-major weights: a [M_total, K], b [G, K, N] (N contiguous),
    other arguments as dg_m_grouped_fp8_gemm_nt_contiguous."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d"); _i32(m_indices, "m_indices")
    M, K = a.shape
    G, Kb, N = b.shape
    _need(Kb == K and tuple(d.shape) == (M, N) and tuple(m_indices.shape) == (M,), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K, G),
          "scale shape mismatch")
    _check("dg_m_grouped_fp8_gemm_nn_contiguous",
           lib.dg_m_grouped_fp8_gemm_nn_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d),
                                                   _ptr(m_indices), M, N, K, G, _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices, stream=None) -> torch.Tensor:
    """Contiguous M-grouped GEMM. a [M_total, K], sfa [KP, ceil4(M_total)], b [G, N, K],
    sfb [G, KP, ceil4(ceil(N/128))], d [M_total, N] bf16, m_indices [M_total] int32 (-1 = pad)."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d"); _i32(m_indices, "m_indices")
    M, K = a.shape
    G, N, Kb = b.shape
    _need(Kb == K and tuple(d.shape) == (M, N) and tuple(m_indices.shape) == (M,), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K, G),
          "scale shape mismatch")
    _check("dg_m_grouped_fp8_gemm_nt_contiguous",
           lib.dg_m_grouped_fp8_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d),
                                                   _ptr(m_indices), M, N, K, G, _stream(stream)))
    return d


def dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, stream=None) -> torch.Tensor:
    """Masked M-grouped GEMM. a [G, max_m, K], sfa [G, KP, ceil4(max_m)], b [G, N, K],
    sfb [G, KP, ceil4(ceil(N/128))], d [G, max_m, N] bf16, masked_m [G] int32 on the device."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d"); _i32(masked_m, "masked_m")
    G, max_m, K = a.shape
    Gb, N, Kb = b.shape
    _need(Gb == G and Kb == K and tuple(d.shape) == (G, max_m, N) and tuple(masked_m.shape) == (G,),
          "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(max_m, K, G) and tuple(sfb.shape) == sf_shape(-(-N // 128), K, G),
          "scale shape mismatch")
    _check("dg_m_grouped_fp8_gemm_nt_masked",
           lib.dg_m_grouped_fp8_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m),
                                               G, max_m, N, K, _stream(stream)))
    return d


# --------------------------------------------------------------------------------------
# FP8 x FP4: b holds packed E2M1 (two per byte, the even element in the low nibble), one
# UE8M0 scale per row per 32 K packed four per int32: sfb [(G,) K/128, ceil4(N)]
# --------------------------------------------------------------------------------------

_FP4_DTYPES = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())


def _fp4(t: torch.Tensor, name: str) -> None:
    _here(t, name)
    _need(t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
    _need(t.dtype in _FP4_DTYPES, f"{name} must hold packed E2M1 bytes (uint8 or float4_e2m1fn_x2)")


def sf_fp4_shape(n: int, k: int, groups: Optional[int] = None):
    """Shape of the FP4 operand's packed scales: [(G,) K/128, ceil4(n)]."""
    shape = (k // 128, 4 * (-(-n // 4)))
    return shape if groups is None else (groups,) + shape


def dg_fp8_fp4_gemm_nt(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A @ B.T with B in FP4. a [M, K] e4m3, sfa [KP, ceil4(M)] int32, b [N, K/2] packed
    E2M1 (32-byte aligned), sfb [K/128, ceil4(N)] int32, c [M, N] bf16 or None, d [M, N] bf16."""
    lib = load_library()
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d")
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] * 2 == K and tuple(d.shape) == (M, N), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_fp4_shape(N, K), "scale shape mismatch")
    if c is not None:
        _bf16(c, "c")
        _need(tuple(c.shape) == (M, N), "c shape mismatch")
    _check("dg_fp8_fp4_gemm_nt", lib.dg_fp8_fp4_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                                        M, N, K, _stream(stream)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices, stream=None) -> torch.Tensor:
    """Contiguous M-grouped FP8 x FP4 GEMM. a [M_total, K], sfa [KP, ceil4(M_total)], b [G, N, K/2]
    packed E2M1, sfb [G, K/128, ceil4(N)], d [M_total, N] bf16, m_indices [M_total] int32 (-1 = pad)."""
    lib = load_library()
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d"); _i32(m_indices, "m_indices")
    M, K = a.shape
    G, N, Kh = b.shape
    _need(Kh * 2 == K and tuple(d.shape) == (M, N) and tuple(m_indices.shape) == (M,), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_fp4_shape(N, K, G), "scale shape mismatch")
    _check("dg_m_grouped_fp8_fp4_gemm_nt_contiguous",
           lib.dg_m_grouped_fp8_fp4_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d),
                                                       _ptr(m_indices), M, N, K, G, _stream(stream)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, stream=None) -> torch.Tensor:
    """Masked M-grouped FP8 x FP4 GEMM. a [G, max_m, K], sfa [G, KP, ceil4(max_m)], b [G, N, K/2]
    packed E2M1, sfb [G, K/128, ceil4(N)], d [G, max_m, N] bf16, masked_m [G] int32 on the device."""
    lib = load_library()
    _fp8(a, "a"); _fp4(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d"); _i32(masked_m, "masked_m")
    G, max_m, K = a.shape
    Gb, N, Kh = b.shape
    _need(Gb == G and Kh * 2 == K and tuple(d.shape) == (G, max_m, N) and tuple(masked_m.shape) == (G,),
          "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(max_m, K, G) and tuple(sfb.shape) == sf_fp4_shape(N, K, G),
          "scale shape mismatch")
    _check("dg_m_grouped_fp8_fp4_gemm_nt_masked",
           lib.dg_m_grouped_fp8_fp4_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m),
                                                   G, max_m, N, K, _stream(stream)))
    return d


def dg_pack_sf_ue8m0(sf: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None,
                     mn_major: bool = False) -> torch.Tensor:
    """FP32 scales [mn, kgroups] (or [kgroups, mn] with mn_major) -> packed UE8M0 int32
    [ceil(kgroups/4), ceil4(mn)] (MN-major)."""
    lib = load_library()
    _here(sf, "sf")
    _need(sf.is_contiguous() and sf.dtype == torch.float32 and sf.dim() == 2,
          "sf must be a contiguous 2-D CUDA float32 tensor")
    mn, kg = (sf.shape[1], sf.shape[0]) if mn_major else (sf.shape[0], sf.shape[1])
    shape = (-(-kg // 4), 4 * (-(-mn // 4)))
    if out is None:
        out = torch.empty(shape, dtype=torch.int32, device=sf.device)
    _i32(out, "out")
    _need(tuple(out.shape) == shape, "out shape mismatch")
    _check("dg_pack_sf_ue8m0", lib.dg_pack_sf_ue8m0(_ptr(sf), _ptr(out), mn, kg, int(mn_major), _stream(stream)))
    return out


# --------------------------------------------------------------------------------------
# Around the GEMMs: norm, router, and the mixture-of-experts layer for a few tokens
# --------------------------------------------------------------------------------------

_TYPES = {torch.bfloat16: 0, torch.float32: 1}      # dg_type
_SCORING = {"softmax": 0, "sigmoid": 1}             # dg_route_scoring
_STREAM_DTYPES = (torch.bfloat16, torch.float32)
_BF16_ONLY, _F32_ONLY, _I32_ONLY = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_FP8_DTYPES = (torch.float8_e4m3fn, torch.uint8)
_MAX_SIZE = 2 ** 31 - 1      # sizes are ints at the C entries, and ctypes would cut off what is above


class _NormDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("H", _I), ("ldx", ctypes.c_size_t), ("ldr", ctypes.c_size_t), ("ldo", ctypes.c_size_t),
                ("residual_type", _I), ("weight_type", _I), ("eps", ctypes.c_float)]


class _RouteDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("E", _I), ("topk", _I), ("ld", ctypes.c_size_t), ("logits_type", _I), ("scoring", _I),
                ("renormalize", _I), ("scale", ctypes.c_float)]


class _BalanceDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("E", _I), ("topk", _I), ("ld", ctypes.c_size_t), ("logits_type", _I), ("scoring", _I),
                ("coef", ctypes.c_float)]


class _RowsDesc(ctypes.Structure):
    _fields_ = [("G", _I), ("M", _I), ("K", _I), ("ldx", ctypes.c_size_t), ("ldg", ctypes.c_size_t), ("x_type", _I)]


# These calls are short (a few microseconds on the device), so their checks read each property of a
# tensor once and build a message only where one fails, and a descriptor is built once for its values.

@functools.lru_cache(maxsize=256)
def _norm_desc(*values):
    return ctypes.byref(_NormDesc(*values))


@functools.lru_cache(maxsize=256)
def _route_desc(*values):
    return ctypes.byref(_RouteDesc(*values))


@functools.lru_cache(maxsize=256)
def _balance_desc(*values):
    return ctypes.byref(_BalanceDesc(*values))


@functools.lru_cache(maxsize=256)
def _rows_desc(*values):
    return ctypes.byref(_RowsDesc(*values))


def _device(t: torch.Tensor, name: str) -> int:
    """The device of a call's first tensor, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        _here(t, name)
    return dev


def _stream_of(stream: Optional[torch.cuda.Stream], dev: int) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _refuse(t: torch.Tensor, name: str, dtypes, shape, dev: int):
    _here(t, name)
    _need(t.get_device() == dev, f"{name} is on another device")
    _need(t.dtype in dtypes, f"{name} must have type {' or '.join(str(d).replace('torch.', '').replace('bfloat16', 'bf16') for d in dtypes)}")
    _need(t.shape == shape, f"{name} shape mismatch: {tuple(t.shape)}, expected {shape}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t: torch.Tensor, name: str, dtypes, shape, dev: int) -> int:
    """Pointer of a contiguous tensor of one of the types and of the shape."""
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _refuse(t, name, dtypes, shape, dev)


def _rows(t: torch.Tensor, name: str, dtypes, shape, dev: int):
    """Pointer and row stride of a 2-D tensor whose columns are contiguous."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        ld, step = t.stride()
        if step != 1 and shape[1] > 1:
            raise ValueError(f"{name} must have contiguous columns")
        return t.data_ptr(), ld if shape[0] > 1 else shape[1]     # of a single row the stride says nothing
    _refuse(t, name, dtypes, shape, dev)


def _two_d(t: torch.Tensor, name: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if shape[0] > _MAX_SIZE or shape[1] > _MAX_SIZE:
        raise ValueError(f"{name} has a size above {_MAX_SIZE}: {tuple(shape)}")
    return shape


def dg_add_rms_norm(x, residual, weight, eps, residual_out=None, y=None, q=None, sf=None, rstd=None, stream=None) -> None:
    """s = x + residual, y = s * rsqrt(mean(s^2) + eps) * weight, and y in E4M3 with a scale per 128
    columns. x [T, H] bf16, residual [T, H] bf16 or float32 (or None), weight [H] bf16 or float32.
    Written where given: residual_out [T, H] = s in residual's type (bf16 or float32 without residual),
    y [T, H] bf16, q [T, H] e4m3 with sf [ceil(H/512), ceil4(T)] int32 (a and sfa of the GEMMs), rstd [T]
    float32. x, residual and residual_out may have strided rows; residual_out may be residual."""
    dev = _device(x, "x")
    T, H = shape = _two_d(x, "x")
    px, ldx = _rows(x, "x", _BF16_ONLY, shape, dev)
    pw = _arg(weight, "weight", _STREAM_DTYPES, (H,), dev)
    pr = po = py = pq = ps = pd = None
    ldr = ldo = H
    rt = torch.bfloat16
    if residual is not None:
        pr, ldr = _rows(residual, "residual", _STREAM_DTYPES, shape, dev)
        rt = residual.dtype
    if residual_out is not None:
        po, ldo = _rows(residual_out, "residual_out", _STREAM_DTYPES, shape, dev)
        _need(residual is None or residual_out.dtype == rt, "residual_out must have residual's type")
        rt = residual_out.dtype
    if y is not None:
        py = _arg(y, "y", _BF16_ONLY, shape, dev)
    if q is not None:
        pq = _arg(q, "q", _FP8_DTYPES, shape, dev)
    if sf is not None:
        ps = _arg(sf, "sf", _I32_ONLY, (-(-H // 512), 4 * (-(-T // 4))), dev)
    if rstd is not None:
        pd = _arg(rstd, "rstd", _F32_ONLY, (T,), dev)
    desc = _norm_desc(T, H, ldx, ldr, ldo, _TYPES[rt], _TYPES[weight.dtype], eps)
    _check("dg_add_rms_norm", (_lib or load_library()).dg_add_rms_norm(px, pr, pw, po, py, pq, ps, pd, desc, _stream_of(stream, dev)))


def dg_add_rms_norm_backward(dy, s, weight, rstd, ds, dx, dresidual, dw, stream=None) -> None:
    """Gradient of dg_add_rms_norm from dy [T, H] bf16 (gradient of y), s [T, H] (its residual_out),
    weight [H], rstd [T] float32 and ds [T, H] of s's type (gradient of residual_out, or None). Writes
    the gradient of s to dx [T, H] bf16 and to dresidual [T, H] of s's type (either may be None), and
    dw [H] float32."""
    dev = _device(dy, "dy")
    T, H = shape = _two_d(dy, "dy")
    pdy = _arg(dy, "dy", _BF16_ONLY, shape, dev)
    ps = _arg(s, "s", _STREAM_DTYPES, shape, dev)
    same = (s.dtype,)
    pw = _arg(weight, "weight", _STREAM_DTYPES, (H,), dev)
    pr = _arg(rstd, "rstd", _F32_ONLY, (T,), dev)
    pds = None if ds is None else _arg(ds, "ds", same, shape, dev)
    pdx = None if dx is None else _arg(dx, "dx", _BF16_ONLY, shape, dev)
    pdr = None if dresidual is None else _arg(dresidual, "dresidual", same, shape, dev)
    pdw = _arg(dw, "dw", _F32_ONLY, (H,), dev)
    _check("dg_add_rms_norm_backward",
           (_lib or load_library()).dg_add_rms_norm_backward(pdy, ps, pw, pr, pds, pdx, pdr, pdw, T, H, _TYPES[s.dtype],
                                                             _TYPES[weight.dtype], _stream_of(stream, dev)))


def _route_args(logits, topk_ids, scoring, renormalize, scale):
    dev = _device(logits, "logits")
    T, E = shape = _two_d(logits, "logits")
    p, ld = _rows(logits, "logits", _STREAM_DTYPES, shape, dev)
    k = _two_d(topk_ids, "topk_ids")[1]
    _need(scoring in _SCORING, "scoring must be softmax or sigmoid")
    desc = _route_desc(T, E, k, ld, _TYPES[logits.dtype], _SCORING[scoring], bool(renormalize), scale)
    return dev, shape, (T, k), p, desc


def dg_moe_route(logits, topk_ids, topk_weights, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """Top-k router: topk_ids [T, k] int32 (largest logit first, ties by lowest index, -1 where no
    unmasked expert is left) and topk_weights [T, k] float32 from logits [T, E] bf16 or float32 (rows may
    be strided; -inf and NaN mask an expert). scoring: "softmax" or "sigmoid"."""
    dev, _, slots, p, desc = _route_args(logits, topk_ids, scoring, renormalize, scale)
    pi = _arg(topk_ids, "topk_ids", _I32_ONLY, slots, dev)
    pw = _arg(topk_weights, "topk_weights", _F32_ONLY, slots, dev)
    _check("dg_moe_route", (_lib or load_library()).dg_moe_route(p, pi, pw, desc, _stream_of(stream, dev)))
    return topk_ids, topk_weights


def dg_moe_route_backward(logits, topk_ids, dweights, dlogits, scoring="softmax", renormalize=True, scale=1.0,
                          stream=None) -> torch.Tensor:
    """Gradient of dg_moe_route: dlogits [T, E] (contiguous, logits' type) from dweights [T, k] float32."""
    dev, shape, slots, p, desc = _route_args(logits, topk_ids, scoring, renormalize, scale)
    pi = _arg(topk_ids, "topk_ids", _I32_ONLY, slots, dev)
    pw = _arg(dweights, "dweights", _F32_ONLY, slots, dev)
    po = _arg(dlogits, "dlogits", (logits.dtype,), shape, dev)
    _check("dg_moe_route_backward", (_lib or load_library()).dg_moe_route_backward(p, pi, pw, po, desc, _stream_of(stream, dev)))
    return dlogits


def _few_tokens(name, fp4, x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, stream):
    dev = _device(x, "x")
    T, H = shape = _two_d(x, "x")
    _need(w13.dim() == 3, "w13 must be 3-D")
    E, N = w13.shape[:2]
    I, k = N // 2, _two_d(topk_ids, "topk_ids")[1]
    per, dtypes = (2, _FP4_DTYPES) if fp4 else (1, _FP8_DTYPES)
    _need(N % 2 == 0 and H % 128 == 0 and I % 128 == 0, "H and I (w13 has 2 I rows) must be multiples of 128")
    if fp4:
        s13, s2 = (E, H // 128, N), (E, I // 128, H)
    else:
        s13, s2 = (E, -(-H // 512), 4 * (-(-N // 512))), (E, -(-I // 512), 4 * (-(-H // 512)))
    px = _arg(x, "x", _FP8_DTYPES, shape, dev)
    psx = _arg(sfx, "sfx", _I32_ONLY, (-(-H // 512), 4 * (-(-T // 4))), dev)
    p13 = _arg(w13, "w13", dtypes, (E, N, H // per), dev)
    ps13 = _arg(sf13, "sf13", _I32_ONLY, s13, dev)
    p2 = _arg(w2, "w2", dtypes, (E, H, I // per), dev)
    ps2 = _arg(sf2, "sf2", _I32_ONLY, s2, dev)
    pi = _arg(topk_ids, "topk_ids", _I32_ONLY, (T, k), dev)
    pw = _arg(topk_weights, "topk_weights", _F32_ONLY, (T, k), dev)
    pc = None if c is None else _arg(c, "c", _BF16_ONLY, shape, dev)
    py = _arg(y, "y", _BF16_ONLY, shape, dev)
    _check(name, getattr(_lib or load_library(), name)(px, psx, p13, ps13, p2, ps2, pi, pw, pc, py, T, k, E, H, I, _stream_of(stream, dev)))
    return y


def dg_moe_fp8_few_tokens(x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, stream=None) -> torch.Tensor:
    """Mixture-of-experts layer for at most 32 tokens: y = c + sum over the slots of weight *
    w2[e] @ (silu(gate) * up), (gate; up) = w13[e] @ x. x [T, H] e4m3 with sfx, w13 [E, 2I, H] e4m3 (gate
    rows first) and w2 [E, H, I] e4m3 with their block scales as for the M-grouped GEMMs, topk_ids [T, k]
    int32 (-1: empty slot), topk_weights [T, k] float32, c [T, H] bf16 or None (may be y), y [T, H] bf16."""
    return _few_tokens("dg_moe_fp8_few_tokens", False, x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, stream)


def dg_moe_fp8_fp4_few_tokens(x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, stream=None) -> torch.Tensor:
    """dg_moe_fp8_few_tokens with the weights in packed E2M1: w13 [E, 2I, H/2] with sf13 [E, H/128, ceil4(2I)],
    w2 [E, H, I/2] with sf2 [E, I/128, ceil4(H)]."""
    return _few_tokens("dg_moe_fp8_fp4_few_tokens", True, x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, stream)


def _balance_args(logits, scoring, coef, topk):
    dev = _device(logits, "logits")
    T, E = shape = _two_d(logits, "logits")
    p, ld = _rows(logits, "logits", _STREAM_DTYPES, shape, dev)
    _need(scoring in _SCORING, "scoring must be softmax or sigmoid")
    return dev, shape, p, _balance_desc(T, E, topk, ld, _TYPES[logits.dtype], _SCORING[scoring], coef)


def dg_moe_balance_loss(logits, topk_ids, counts, live_rows, prob_mean, loss, scoring="softmax", coef=1.0, stream=None):
    """Balance loss of a router: with p the probabilities of each row of logits [T, E] bf16 or float32 (rows may be
    strided; -inf and NaN mask an expert; softmax, or sigmoids divided by their sum) and f the experts' shares of the
    slots of topk_ids [T, k] int32, loss [1] float32 = coef * E * sum(f * mean of p over the live rows). Also writes
    counts [E] int32 (slots per expert), live_rows [1] int32 and prob_mean [E] float32. Returns loss."""
    k = _two_d(topk_ids, "topk_ids")[1]
    dev, (T, E), p, desc = _balance_args(logits, scoring, coef, k)
    pi = _arg(topk_ids, "topk_ids", _I32_ONLY, (T, k), dev)
    pc = _arg(counts, "counts", _I32_ONLY, (E,), dev)
    pl = _arg(live_rows, "live_rows", _I32_ONLY, (1,), dev)
    pm = _arg(prob_mean, "prob_mean", _F32_ONLY, (E,), dev)
    po = _arg(loss, "loss", _F32_ONLY, (1,), dev)
    _check("dg_moe_balance_loss", (_lib or load_library()).dg_moe_balance_loss(p, pi, pc, pl, pm, po, desc, _stream_of(stream, dev)))
    return loss


def dg_moe_balance_loss_backward(logits, counts, live_rows, dloss, dlogits, base=None, scoring="softmax", coef=1.0,
                                 stream=None) -> torch.Tensor:
    """Gradient of dg_moe_balance_loss with respect to logits, plus `base`: dlogits [T, E] (contiguous, logits' type)
    from the forward call's counts [E] and live_rows [1] and dloss [1] float32. base [T, E] of logits' type (the
    gradient by other paths, or None) may be dlogits."""
    dev, (T, E), p, desc = _balance_args(logits, scoring, coef, 1)
    same = (logits.dtype,)
    pc = _arg(counts, "counts", _I32_ONLY, (E,), dev)
    pl = _arg(live_rows, "live_rows", _I32_ONLY, (1,), dev)
    pd = _arg(dloss, "dloss", _F32_ONLY, (1,), dev)
    pb = None if base is None else _arg(base, "base", same, (T, E), dev)
    po = _arg(dlogits, "dlogits", same, (T, E), dev)
    _check("dg_moe_balance_loss_backward",
           (_lib or load_library()).dg_moe_balance_loss_backward(p, pc, pl, pd, pb, po, desc, _stream_of(stream, dev)))
    return dlogits


# --------------------------------------------------------------------------------------
# FP4: quantisation of rows, and the GEMMs of two FP4 operands. Packed E2M1 and scales as above
# --------------------------------------------------------------------------------------

def _fp4_rows(x, per, dtypes, masked_m):
    """Device, leading shape, rows, result columns, pointers of x and masked_m, descriptor."""
    dev = _device(x, "x")
    shape, strides = x.shape, x.stride()
    grouped = len(shape) == 3
    if not grouped and len(shape) != 2:
        raise ValueError("x must be [M, K] or [G, M, K]")
    if x.dtype not in dtypes:
        raise ValueError(f"x must have type {' or '.join(str(d).replace('torch.', '') for d in dtypes)}")
    M, C = shape[-2:]
    G = shape[0] if grouped else 1
    if G > _MAX_SIZE or M > _MAX_SIZE or C > _MAX_SIZE:
        raise ValueError(f"x has a size above {_MAX_SIZE}: {tuple(shape)}")
    if strides[-1] != 1:
        raise ValueError("x must have contiguous columns")
    if C % (128 * per):
        raise ValueError(f"x must have a multiple of {128 * per} columns")
    pm = None
    if masked_m is not None:
        _need(grouped, "masked_m needs x with groups, [G, M, K]")
        pm = _arg(masked_m, "masked_m", _I32_ONLY, (G,), dev)
    desc = _rows_desc(G, M, C // per, strides[-2] if M > 1 else C, strides[0] if G > 1 else 0, _TYPES[x.dtype])
    return dev, shape[:1] if grouped else (), M, C // per, x.data_ptr(), pm, desc


def _quantize(name, per, dtypes, x, q, sf, masked_m, stream):
    dev, lead, M, K, px, pm, desc = _fp4_rows(x, per, dtypes, masked_m)
    pq = _arg(q, "q", _FP4_DTYPES, (*lead, M, K // 2), dev)
    ps = _arg(sf, "sf", _I32_ONLY, (*lead, K // 128, 4 * (-(-M // 4))), dev)
    _check(name, getattr(_lib or load_library(), name)(px, pm, pq, ps, desc, _stream_of(stream, dev)))
    return q, sf


def dg_quantize_fp4(x, q, sf, masked_m=None, stream=None):
    """Rows to FP4: x [M, K] or [G, M, K] bf16 or float32 (rows and groups may be strided) -> q [.., M, K/2] packed
    E2M1 and sf [.., K/128, ceil4(M)] int32, one UE8M0 scale per row per 32 columns: the operands of the FP4 GEMMs and
    the FP4 weights of the FP8 x FP4 ones. With masked_m [G] int32 on the device only the first masked_m[g] rows of each
    group are read and written."""
    return _quantize("dg_quantize_fp4", 1, _STREAM_DTYPES, x, q, sf, masked_m, stream)


def dg_swiglu_quantize_fp4(x, q, sf, masked_m=None, stream=None):
    """dg_quantize_fp4 of silu(gate) * up, for x [M, 2K] or [G, M, 2K] bf16 whose first K columns are the gate and
    last K columns up."""
    return _quantize("dg_swiglu_quantize_fp4", 2, _BF16_ONLY, x, q, sf, masked_m, stream)


def dg_swiglu_backward(x, dy, dx, masked_m=None, stream=None) -> torch.Tensor:
    """Gradient of silu(gate) * up: dx [.., M, 2K] bf16 from x [.., M, 2K] (gate | up; rows may be strided) and dy
    [.., M, K] bf16. dx may be x where x is contiguous. Rows behind masked_m are not written."""
    dev, lead, M, K, px, pm, desc = _fp4_rows(x, 2, _BF16_ONLY, masked_m)
    pd = _arg(dy, "dy", _BF16_ONLY, (*lead, M, K), dev)
    po = _arg(dx, "dx", _BF16_ONLY, (*lead, M, 2 * K), dev)
    _check("dg_swiglu_backward", (_lib or load_library()).dg_swiglu_backward(px, pd, pm, po, desc, _stream_of(stream, dev)))
    return dx


def _sizes(*sizes):
    if max(sizes) > _MAX_SIZE:
        raise ValueError(f"a size is above {_MAX_SIZE}: {max(sizes)}")


def dg_fp4_gemm_nt(a, sfa, b, sfb, c, d, stream=None) -> torch.Tensor:
    """D = C + A @ B.T of two FP4 operands. a [M, K/2] packed E2M1 with sfa [K/128, ceil4(M)] int32, b [N, K/2] with
    sfb [K/128, ceil4(N)], c [M, N] bf16 or None (may be d), d [M, N] bf16 (written)."""
    dev = _device(a, "a")
    M, Kh = _two_d(a, "a")
    N = _two_d(b, "b")[0]
    _sizes(2 * Kh, N)
    pa = _arg(a, "a", _FP4_DTYPES, (M, Kh), dev)
    pb = _arg(b, "b", _FP4_DTYPES, (N, Kh), dev)
    psa = _arg(sfa, "sfa", _I32_ONLY, sf_fp4_shape(M, 2 * Kh), dev)
    psb = _arg(sfb, "sfb", _I32_ONLY, sf_fp4_shape(N, 2 * Kh), dev)
    pc = None if c is None else _arg(c, "c", _BF16_ONLY, (M, N), dev)
    pd = _arg(d, "d", _BF16_ONLY, (M, N), dev)
    _check("dg_fp4_gemm_nt", (_lib or load_library()).dg_fp4_gemm_nt(pa, psa, pb, psb, pc, pd, M, N, 2 * Kh, _stream_of(stream, dev)))
    return d


def dg_m_grouped_fp4_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices, stream=None) -> torch.Tensor:
    """Contiguous M-grouped FP4 GEMM: a [M_total, K/2] packed E2M1, sfa [K/128, ceil4(M_total)], b [G, N, K/2], sfb
    [G, K/128, ceil4(N)], d [M_total, N] bf16, m_indices [M_total] int32 (-1 = pad)."""
    dev = _device(a, "a")
    M, Kh = _two_d(a, "a")
    _need(b.dim() == 3, "b must be 3-D")
    G, N = b.shape[:2]
    _sizes(2 * Kh, G, N)
    pa = _arg(a, "a", _FP4_DTYPES, (M, Kh), dev)
    pb = _arg(b, "b", _FP4_DTYPES, (G, N, Kh), dev)
    psa = _arg(sfa, "sfa", _I32_ONLY, sf_fp4_shape(M, 2 * Kh), dev)
    psb = _arg(sfb, "sfb", _I32_ONLY, sf_fp4_shape(N, 2 * Kh, G), dev)
    pd = _arg(d, "d", _BF16_ONLY, (M, N), dev)
    pi = _arg(m_indices, "m_indices", _I32_ONLY, (M,), dev)
    _check("dg_m_grouped_fp4_gemm_nt_contiguous",
           (_lib or load_library()).dg_m_grouped_fp4_gemm_nt_contiguous(pa, psa, pb, psb, pd, pi, M, N, 2 * Kh, G, _stream_of(stream, dev)))
    return d


def dg_m_grouped_fp4_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, stream=None) -> torch.Tensor:
    """Masked M-grouped FP4 GEMM: a [G, max_m, K/2] packed E2M1, sfa [G, K/128, ceil4(max_m)], b [G, N, K/2], sfb
    [G, K/128, ceil4(N)], d [G, max_m, N] bf16, masked_m [G] int32 on the device."""
    dev = _device(a, "a")
    _need(a.dim() == 3 and b.dim() == 3, "a and b must be 3-D")
    G, max_m, Kh = a.shape
    N = b.shape[1]
    _sizes(2 * Kh, G, N, max_m)
    pa = _arg(a, "a", _FP4_DTYPES, (G, max_m, Kh), dev)
    pb = _arg(b, "b", _FP4_DTYPES, (G, N, Kh), dev)
    psa = _arg(sfa, "sfa", _I32_ONLY, sf_fp4_shape(max_m, 2 * Kh, G), dev)
    psb = _arg(sfb, "sfb", _I32_ONLY, sf_fp4_shape(N, 2 * Kh, G), dev)
    pd = _arg(d, "d", _BF16_ONLY, (G, max_m, N), dev)
    pm = _arg(masked_m, "masked_m", _I32_ONLY, (G,), dev)
    _check("dg_m_grouped_fp4_gemm_nt_masked",
           (_lib or load_library()).dg_m_grouped_fp4_gemm_nt_masked(pa, psa, pb, psb, pd, pm, G, max_m, N, 2 * Kh, _stream_of(stream, dev)))
    return d


def dg_get_mk_alignment_for_contiguous_layout() -> int:
    return load_library().dg_get_mk_alignment_for_contiguous_layout()


def dg_set_mk_alignment_for_contiguous_layout(alignment: int) -> None:
    """Set the segment alignment callers are told to pad to (a positive multiple of 128)."""
    _check("dg_set_mk_alignment_for_contiguous_layout",
           load_library().dg_set_mk_alignment_for_contiguous_layout(int(alignment)))


def dg_get_theoretical_mk_alignment_for_contiguous_layout() -> int:
    return load_library().dg_get_theoretical_mk_alignment_for_contiguous_layout()


def dg_get_tma_aligned_size(mn: int, elem_bytes: int) -> int:
    return load_library().dg_get_tma_aligned_size(mn, elem_bytes)


def dg_set_num_sms(n: int) -> None:
    _check("dg_set_num_sms", load_library().dg_set_num_sms(n))


def dg_get_num_sms() -> int:
    return load_library().dg_get_num_sms()


def dg_reserve_workspace(nbytes: int, stream=None) -> None:
    """Reserve (at least nbytes of) the library's workspace for the stream (current by default)."""
    _check("dg_reserve_workspace", load_library().dg_reserve_workspace(_stream(stream), nbytes))


def dg_release_workspace(stream=None) -> None:
    _check("dg_release_workspace", load_library().dg_release_workspace(_stream(stream)))


def dg_get_workspace_size(stream=None) -> int:
    return int(load_library().dg_get_workspace_size(_stream(stream)))


def dg_set_pdl(enable: bool) -> None:
    """Programmatic dependent launch on (True) or off (False) for later launches."""
    _check("dg_set_pdl", load_library().dg_set_pdl(1 if enable else 0))


def dg_get_pdl() -> bool:
    return bool(load_library().dg_get_pdl())


def dg_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device-side error status code."""
    return load_library().dg_get_device_status(_stream(stream))


def dg_status_string(status: int) -> str:
    return load_library().dg_status_string(status).decode()


def dg_last_cuda_error() -> int:
    """The last CUDA error code the library saw on this host thread (0 if none)."""
    return load_library().dg_last_cuda_error()


def dg_set_debug(fault_mode: int, wait_timeout_ns: int = 0) -> None:
    """Failure-detection test hook: fault_mode 1 makes later launches time out on purpose
    (their producer issues nothing); wait_timeout_ns bounds every pipeline wait (0 = 2 s)."""
    _check("dg_set_debug", load_library().dg_set_debug(fault_mode, wait_timeout_ns))


def dg_measure_fp8_mma_tflops(iters_per_sm: int = 4096) -> tuple[float, float]:
    """Measured FP8 tensor-core ceiling of the current device: (TFLOP/s, kernel ms) of an
    MMA-only kernel (block-scaled 128 x 256 x 32 MMAs from shared memory on every SM)."""
    tf, ms = ctypes.c_double(0.0), ctypes.c_double(0.0)
    _check("dg_measure_fp8_mma_tflops",
           load_library().dg_measure_fp8_mma_tflops(int(iters_per_sm), ctypes.byref(tf), ctypes.byref(ms)))
    return tf.value, ms.value


def dg_fp8_gemm_nt_no_alloc(a, sfa, b, sfb, c, d, status, stream=None) -> torch.Tensor:
    """D = C + A @ B.T without any device allocation by the library, for callers that
    cannot allocate at call time (graph capture, fixed-footprint servers, custom
    allocators). Same tensors as dg_fp8_gemm_nt plus `status`, a CUDA uint32/int32 tensor
    of one element that receives device-side error bits. The library's fixed 16 MiB
    scratch bounds the problem size (DG_ERR_INVALID_ARG beyond it); calls that overlap on
    the GPU race on that scratch."""
    lib = load_library()
    _fp8(a, "a"); _fp8(b, "b"); _i32(sfa, "sfa"); _i32(sfb, "sfb"); _bf16(d, "d")
    _here(status, "status")
    _need(status.numel() == 1 and status.element_size() == 4, "status must be one 4-byte CUDA word")
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K and tuple(d.shape) == (M, N), "shape mismatch")
    _need(tuple(sfa.shape) == sf_shape(M, K) and tuple(sfb.shape) == sf_shape(-(-N // 128), K), "scale shape mismatch")
    if c is not None:
        _bf16(c, "c")
        _need(tuple(c.shape) == (M, N), "c shape mismatch")
    _check("dg_fp8_gemm_nt_no_alloc",
           lib.dg_fp8_gemm_nt_no_alloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d), _ptr(status),
                                       M, N, K, _stream(stream)))
    return d
