"""Block-scaled FP8 GEMM and MoE grouped GEMM for GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/dg.h`` (``libdg.so``, built in-tree by
``build.py``). The functions carry the C names and only marshal arguments: torch tensors provide
device memory and the current CUDA stream; every step of the computation runs in the library's CUDA
kernels. There is no fallback: when the library or a supported GPU is missing, calls raise.

Operation (DeepGEMM pages, "DeepSeek DeepGEMM" usage example and feature list):
``D[m,n] = sum_kb sfa[m,kb] * sfb[n//128,kb] * sum_{k in block kb} A[m,k] B[n,k]`` with e4m3 A/B,
FP32 1x128 (A) and 128x128 (B) block scales, BF16 output; plus the m-grouped contiguous and masked
layouts and the k-grouped FP32 weight gradient. Around them: the router, a whole MoE layer for a few
tokens, and the GEMM with bias, activation and residual in its epilogue, with its backward pass.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

__all__ = [
    "DGError", "load", "dg_gemm_fp8_nt", "dg_gemm_fp8", "dg_gemm_fp8_nt_ue8m0", "dg_gemm_fp8_nt_ue8m0_packed",
    "dg_m_grouped_contiguous", "dg_m_grouped_masked",
    "dg_k_grouped_wgrad", "dg_wgrad_fp8_nt", "dg_gemm_fp8_nt_epilogue", "dg_epilogue_backward",
    "dg_moe_route", "dg_moe_route_backward", "dg_moe_layer",
    "epilogue_backward_workspace", "moe_layer_workspace", "ACTIVATIONS", "SCORES",
    "dg_device_status", "dg_status_string", "scale_shapes", "library_path",
    "TUNE_KNOBS", "dg_tuning_set", "dg_tuning_get", "dg_tuning_reset", "tuning", "dg_testing_arm_wait_timeout",
    "FAULTS", "dg_testing_arm_fault",
]

_lock = threading.Lock()
_lib = None

DG_OK = 0
STATUS_NAMES = {0: "DG_OK", 1: "DG_INVALID_ARG", 2: "DG_UNSUPPORTED_SHAPE", 3: "DG_MISALIGNED",
                4: "DG_CUDA_ERROR", 5: "DG_NO_DEVICE_SUPPORT", 6: "DG_DEVICE_TIMEOUT", 7: "DG_SCALE_NOT_UE8M0"}


class DGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


def library_path() -> str:
    from . import build as _build
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load ``libdg.so`` (building it with nvcc first when absent or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            from . import build as _build
            path = _build.build() if build_if_missing else _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libdg.so not found at {path}; run moe_grouped_gemm_tma_gb300/build.py")
            L = ctypes.CDLL(path)
            P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64
            L.dg_gemm_fp8_nt.argtypes = [P, P, P, P, P, I, I, I, P]
            L.dg_gemm_fp8.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
            L.dg_gemm_fp8_nt_ue8m0.argtypes = [P, P, P, P, P, I, I, I, P]
            L.dg_gemm_fp8_nt_ue8m0_packed.argtypes = [P, P, P, P, P, I, I, I, P]
            L.dg_m_grouped_contiguous.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
            L.dg_m_grouped_masked.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
            L.dg_k_grouped_wgrad.argtypes = [P, P, P, P, P, P, I, I, I, P]
            L.dg_wgrad_fp8_nt.argtypes = [P, P, P, P, P, I, I, I, I, P]
            L.dg_gemm_fp8_nt_epilogue.argtypes = [P, P, P, P, P, P, I, P, P, I, I, I, P]
            L.dg_epilogue_backward.argtypes = [P, P, I, P, P, P, P, P, P, S, I, I, P]
            L.dg_moe_route.argtypes = [P, I, P, P, P, I, I, I, I, I, F, P]
            L.dg_moe_route_backward.argtypes = [P, I, P, P, P, I, I, I, I, I, F, P]
            L.dg_moe_layer.argtypes = [P, P, P, P, P, P, P, P, P, P, S, I, I, I, I, I, I, P]
            L.dg_epilogue_backward_workspace.argtypes = [I, I]
            L.dg_moe_layer_workspace.argtypes = [I, I, I, I, I]
            L.dg_epilogue_backward_workspace.restype = L.dg_moe_layer_workspace.restype = S
            L.dg_device_status.argtypes = [P]
            L.dg_tuning_set.argtypes = [I, I]
            L.dg_tuning_set.restype = I
            L.dg_tuning_get.argtypes = [I]
            L.dg_tuning_get.restype = I
            L.dg_tuning_reset.argtypes = []
            L.dg_tuning_reset.restype = None
            L.dg_testing_arm_wait_timeout.argtypes = [ctypes.c_uint64]
            L.dg_testing_arm_wait_timeout.restype = I
            L.dg_testing_arm_fault.argtypes = [I, ctypes.c_uint64]
            L.dg_testing_arm_fault.restype = I
            L.dg_status_string.argtypes = [I]
            L.dg_status_string.restype = ctypes.c_char_p
            for f in ("dg_gemm_fp8_nt", "dg_gemm_fp8", "dg_gemm_fp8_nt_ue8m0", "dg_gemm_fp8_nt_ue8m0_packed",
                      "dg_m_grouped_contiguous", "dg_m_grouped_masked",
                      "dg_k_grouped_wgrad", "dg_wgrad_fp8_nt", "dg_gemm_fp8_nt_epilogue", "dg_epilogue_backward",
                      "dg_moe_route", "dg_moe_route_backward", "dg_moe_layer", "dg_device_status"):
                getattr(L, f).restype = I
            _lib = L
    return _lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


# The calls of a decode step are a few microseconds of GPU work each, so what the binding does per call is kept
# small: addresses go to ctypes as plain numbers, and the current stream is asked for as one (building a
# torch Stream object for it takes 3 us).
def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream):
    if stream is None:
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _codes(t, name):
    torch = _torch()
    if t.dtype != torch.float8_e4m3fn and t.dtype != torch.uint8:
        raise TypeError(f"{name} must hold e4m3 codes (torch.float8_e4m3fn or uint8), got {t.dtype}")
    return _dense(t, name)


def _dense(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32(t, name):
    torch = _torch()
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _dense(t, name)


def _check(status: int, where: str):
    if status != DG_OK:
        raise DGError(status, where)


def scale_shapes(M: int, N: int, K: int):
    """Shapes of (sfa, sfb) for a normal GEMM: ([M, K/128], [ceil(N/128), K/128])."""
    return (M, K // 128), ((N + 127) // 128, K // 128)


def dg_gemm_fp8_nt(A, sfa, B, sfb, D, stream=None):
    """D[M,N] (bf16) = A[M,K] . B[N,K]^T with sfa [M,K/128] and sfb [ceil(N/128),K/128] scales."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    D = _dense(D, "D")
    if D.dtype != torch.bfloat16:
        raise TypeError("D must be bfloat16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} D {tuple(D.shape)}")
    if (tuple(sfa.shape), tuple(sfb.shape)) != scale_shapes(M, N, K):
        raise ValueError(f"scale shapes {tuple(sfa.shape)}, {tuple(sfb.shape)} != {scale_shapes(M, N, K)}")
    st = load().dg_gemm_fp8_nt(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(D), M, N, K, _stream(stream))
    _check(st, "dg_gemm_fp8_nt")
    return D


def dg_gemm_fp8(A, sfa, B, sfb, D, a_mn_major=False, b_mn_major=False, stream=None):
    """The normal GEMM for any operand layout: A stored [M,K] or (a_mn_major) [K,M]; B stored [N,K] or
    (b_mn_major) [K,N]; same scales and output as dg_gemm_fp8_nt."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    D = _dense(D, "D")
    if D.dtype != torch.bfloat16:
        raise TypeError("D must be bfloat16")
    K, M = A.shape if a_mn_major else A.shape[::-1]
    KB, N = B.shape if b_mn_major else B.shape[::-1]
    if KB != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} D {tuple(D.shape)}")
    if (tuple(sfa.shape), tuple(sfb.shape)) != scale_shapes(M, N, K):
        raise ValueError(f"scale shapes {tuple(sfa.shape)}, {tuple(sfb.shape)} != {scale_shapes(M, N, K)}")
    st = load().dg_gemm_fp8(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(D), M, N, K,
                            1 if a_mn_major else 0, 1 if b_mn_major else 0, _stream(stream))
    _check(st, "dg_gemm_fp8")
    return D


def dg_gemm_fp8_nt_ue8m0(A, sfa, B, sfb, D, stream=None):
    """dg_gemm_fp8_nt for power-of-two scales on the block-scaled (UE8M0) tensor-core path."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    D = _dense(D, "D")
    if D.dtype != torch.bfloat16:
        raise TypeError("D must be bfloat16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} D {tuple(D.shape)}")
    if (tuple(sfa.shape), tuple(sfb.shape)) != scale_shapes(M, N, K):
        raise ValueError(f"scale shapes {tuple(sfa.shape)}, {tuple(sfb.shape)} != {scale_shapes(M, N, K)}")
    st = load().dg_gemm_fp8_nt_ue8m0(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(D), M, N, K, _stream(stream))
    _check(st, "dg_gemm_fp8_nt_ue8m0")
    return D


def dg_gemm_fp8_nt_ue8m0_packed(A, sfa, B, sfb, D, stream=None):
    """The block-scaled GEMM with packed UE8M0 scales: sfa int32 [M, ceil(K/512)], sfb int32
    [ceil(N/128), ceil(K/512)], byte j of word w = biased exponent of K block 4w + j."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb, D = _dense(sfa, "sfa"), _dense(sfb, "sfb"), _dense(D, "D")
    if sfa.dtype != torch.int32 or sfb.dtype != torch.int32:
        raise TypeError("packed scales must be int32")
    if D.dtype != torch.bfloat16:
        raise TypeError("D must be bfloat16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(D.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)} B {tuple(B.shape)} D {tuple(D.shape)}")
    words = (K // 128 + 3) // 4
    if tuple(sfa.shape) != (M, words) or tuple(sfb.shape) != ((N + 127) // 128, words):
        raise ValueError(f"packed scale shapes {tuple(sfa.shape)}, {tuple(sfb.shape)} != {(M, words)}, {((N + 127) // 128, words)}")
    st = load().dg_gemm_fp8_nt_ue8m0_packed(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(D), M, N, K, _stream(stream))
    _check(st, "dg_gemm_fp8_nt_ue8m0_packed")
    return D


def dg_m_grouped_contiguous(A, sfa, B, sfb, m_indices, D, stream=None):
    """Contiguous-layout grouped GEMM: D[r] = A[r] . B[m_indices[r]]^T (bf16); A [Mt,K], B [G,N,K]."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    m_indices, D = _dense(m_indices, "m_indices"), _dense(D, "D")
    if m_indices.dtype != torch.int32 or D.dtype != torch.bfloat16:
        raise TypeError("m_indices must be int32 and D bfloat16")
    Mt, K = A.shape
    G, N, K2 = B.shape
    if K2 != K or tuple(D.shape) != (Mt, N) or m_indices.numel() != Mt:
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (Mt, K // 128) or tuple(sfb.shape) != (G, (N + 127) // 128, K // 128):
        raise ValueError("scale shape mismatch")
    st = load().dg_m_grouped_contiguous(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(m_indices), _ptr(D),
                                        Mt, N, K, G, _stream(stream))
    _check(st, "dg_m_grouped_contiguous")
    return D


def dg_m_grouped_masked(A, sfa, B, sfb, masked_m, D, expected_m: int = 0, stream=None):
    """Masked-layout grouped GEMM: D[g,r] = A[g,r] . B[g]^T for r < masked_m[g]; other rows untouched."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    masked_m, D = _dense(masked_m, "masked_m"), _dense(D, "D")
    if masked_m.dtype != torch.int32 or D.dtype != torch.bfloat16:
        raise TypeError("masked_m must be int32 and D bfloat16")
    G, max_m, K = A.shape
    G2, N, K2 = B.shape
    if G2 != G or K2 != K or tuple(D.shape) != (G, max_m, N) or masked_m.numel() != G:
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (G, max_m, K // 128) or tuple(sfb.shape) != (G, (N + 127) // 128, K // 128):
        raise ValueError("scale shape mismatch")
    st = load().dg_m_grouped_masked(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(masked_m), _ptr(D),
                                    G, max_m, N, K, int(expected_m), _stream(stream))
    _check(st, "dg_m_grouped_masked")
    return D


def dg_k_grouped_wgrad(A, sfa, B, sfb, ks, D, stream=None):
    """k-grouped FP32 weight gradient: D[g] += A[:, win_g] . B[:, win_g]^T, windows of widths ``ks``."""
    torch = _torch()
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    D = _f32(D, "D")
    ks_list = [int(k) for k in (ks.tolist() if hasattr(ks, "tolist") else ks)]
    G = len(ks_list)
    M, sumK = A.shape
    N = B.shape[0]
    if B.shape[1] != sumK or sum(ks_list) != sumK or tuple(D.shape) != (G, M, N):
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (M, sumK // 128) or tuple(sfb.shape) != (N, sumK // 128):
        raise ValueError("scale shape mismatch")
    ks_arr = (ctypes.c_int32 * max(G, 1))(*ks_list)
    st = load().dg_k_grouped_wgrad(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), ks_arr, _ptr(D), G, M, N,
                                   _stream(stream))
    _check(st, "dg_k_grouped_wgrad")
    return D


def dg_wgrad_fp8_nt(A, sfa, B, sfb, D, accumulate=True, stream=None):
    """Dense FP32 weight gradient: D += A . B^T (accumulate) or D = A . B^T, 1x128 scales on both."""
    A, B = _codes(A, "A"), _codes(B, "B")
    sfa, sfb = _f32(sfa, "sfa"), _f32(sfb, "sfb")
    D = _f32(D, "D")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(D.shape) != (M, N):
        raise ValueError("shape mismatch")
    if tuple(sfa.shape) != (M, K // 128) or tuple(sfb.shape) != (N, K // 128):
        raise ValueError("scale shape mismatch")
    st = load().dg_wgrad_fp8_nt(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(D), M, N, K,
                                1 if accumulate else 0, _stream(stream))
    _check(st, "dg_wgrad_fp8_nt")
    return D


# Activations and router scores by name (include/dg.h).
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
SCORES = {"softmax": 0, "sigmoid": 1}


def _choice(table, name, what):
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}, got {name!r}")
    return table[name]


def _refuse(**args):
    """The checks that a call's arguments have not passed, one by one, so that the first that fails says what is
    wrong: name=(tensor or None, dtypes, shape or None)."""
    for name, (t, dtypes, shape) in args.items():
        if t is None:
            continue
        if t.dtype not in dtypes:
            if _torch().uint8 in dtypes and len(dtypes) == 2:
                _codes(t, name)
            raise TypeError(f"{name} must be {' or '.join(str(d).replace('torch.', '') for d in dtypes)}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)} (shape mismatch)")
        _dense(t, name)


def _bytes(t, name):
    """A workspace's address and size."""
    torch = _torch()
    if t is None:
        return None, 0
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8, got {t.dtype}")
    return _ptr(_dense(t, name)), t.numel()


# The five functions below check what the others do, but in one expression: a decode step makes these calls for
# a few microseconds of GPU work each, and a helper's call per argument adds up to as much. Only arguments that
# do not pass are looked at one by one.
def _good(t, dtype, shape):
    return t is None or (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous())


def dg_gemm_fp8_nt_epilogue(A, sfa, B, sfb, D, bias=None, act="none", residual=None, Z=None, stream=None):
    """D = act(A . B^T + bias) + residual (bf16); A, sfa, B, sfb as dg_gemm_fp8_nt, bias fp32 [N], residual bf16
    [M,N] (may be D), Z bf16 [M,N] receives the pre-activation."""
    torch = _torch_module or _torch()
    bf16, f32, e4m3 = torch.bfloat16, torch.float32, (torch.float8_e4m3fn, torch.uint8)
    M, K = A.shape
    N = B.shape[0]
    MN = (M, N)
    if not (A.dtype in e4m3 and B.dtype in e4m3 and sfa.dtype is f32 and sfb.dtype is f32 and D.dtype is bf16
            and B.shape[1] == K and sfa.shape == (M, K // 128) and sfb.shape == ((N + 127) // 128, K // 128) and D.shape == MN
            and A.is_cuda and A.is_contiguous() and B.is_cuda and B.is_contiguous() and sfa.is_cuda and sfa.is_contiguous()
            and sfb.is_cuda and sfb.is_contiguous() and D.is_cuda and D.is_contiguous()
            and (bias is None or _good(bias, f32, (N,))) and (residual is None or _good(residual, bf16, MN))
            and (Z is None or _good(Z, bf16, MN))):
        _refuse(A=(A, e4m3, None), B=(B, e4m3, (N, K)), sfa=(sfa, (f32,), (M, K // 128)), sfb=(sfb, (f32,), ((N + 127) // 128, K // 128)),
                D=(D, (bf16,), MN), bias=(bias, (f32,), (N,)), residual=(residual, (bf16,), MN), Z=(Z, (bf16,), MN))
    st = (_lib or load()).dg_gemm_fp8_nt_epilogue(
        A.data_ptr(), sfa.data_ptr(), B.data_ptr(), sfb.data_ptr(), D.data_ptr(), None if bias is None else bias.data_ptr(),
        _choice(ACTIVATIONS, act, "act"), None if residual is None else residual.data_ptr(), None if Z is None else Z.data_ptr(),
        M, N, K, _stream(stream))
    if st:
        raise DGError(st, "dg_gemm_fp8_nt_epilogue")
    return D


# What a workspace's first call expects to be zero, from its start (include/dg.h); the rest is written before it is read.
_EPILOGUE_BACKWARD_ZEROED, _MOE_LAYER_ZEROED = 1024, 4096


def _workspace(size, zeroed, device):
    torch = _torch()
    ws = torch.empty(size, dtype=torch.uint8, device=device or "cuda")
    ws[:zeroed].zero_()
    return ws


def epilogue_backward_workspace(M: int, N: int, device=None):
    """A workspace for dg_epilogue_backward with dbias at up to this size, ready for its first call."""
    return _workspace(load().dg_epilogue_backward_workspace(M, N), _EPILOGUE_BACKWARD_ZEROED, device)


def dg_epilogue_backward(dD, Z, q, sf, qt, sft, dbias, workspace=None, act="none", stream=None):
    """dZ = dD * act'(Z), bf16 [M,N] in, out as e4m3 codes q [M,N] with scales sf [M,N/128], codes of the
    transpose qt [N,Mp] with scales sft [N,Mp/128] (Mp = M rounded up to 128), and dbias fp32 [N], the sum of
    its rows. q with sf, qt with sft, and dbias may be None; dbias needs a workspace
    (epilogue_backward_workspace). Z is not read for act "none"."""
    torch = _torch_module or _torch()
    bf16, f32, e4m3 = torch.bfloat16, torch.float32, (torch.float8_e4m3fn, torch.uint8)
    M, N = dD.shape
    Mp = (M + 127) // 128 * 128
    MN = (M, N)
    if not (dD.dtype is bf16 and dD.is_cuda and dD.is_contiguous() and (Z is None or _good(Z, bf16, MN))
            and (q is None or (q.dtype in e4m3 and q.shape == MN and q.is_cuda and q.is_contiguous()))
            and (qt is None or (qt.dtype in e4m3 and qt.shape == (N, Mp) and qt.is_cuda and qt.is_contiguous()))
            and (sf is None or _good(sf, f32, (M, N // 128))) and (sft is None or _good(sft, f32, (N, Mp // 128)))
            and (dbias is None or _good(dbias, f32, (N,)))):
        _refuse(dD=(dD, (bf16,), None), Z=(Z, (bf16,), MN), q=(q, e4m3, MN), qt=(qt, e4m3, (N, Mp)), sf=(sf, (f32,), (M, N // 128)),
                sft=(sft, (f32,), (N, Mp // 128)), dbias=(dbias, (f32,), (N,)))
    ws, size = _bytes(workspace, "workspace")
    st = (_lib or load()).dg_epilogue_backward(
        dD.data_ptr(), None if Z is None else Z.data_ptr(), _choice(ACTIVATIONS, act, "act"), None if q is None else q.data_ptr(),
        None if sf is None else sf.data_ptr(), None if qt is None else qt.data_ptr(), None if sft is None else sft.data_ptr(),
        None if dbias is None else dbias.data_ptr(), ws, size, M, N, _stream(stream))
    if st:
        raise DGError(st, "dg_epilogue_backward")


def dg_moe_route(logits, ids, weights, bias=None, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """The router: ids int32 [T,k] and weights fp32 [T,k] of the k largest selection values of each row of
    logits [T,E] (bf16 or fp32; with a bias fp32 [E], sigmoid scoring only, sigmoid(logit) + bias)."""
    torch = _torch_module or _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    T, E = logits.shape
    k = ids.shape[1]
    kind = logits.dtype
    Tk = (T, k)
    if not ((kind is f32 or kind is bf16) and logits.is_cuda and logits.is_contiguous() and ids.dtype is torch.int32 and ids.shape == Tk
            and ids.is_cuda and ids.is_contiguous() and weights.dtype is f32 and weights.shape == Tk and weights.is_cuda
            and weights.is_contiguous() and (bias is None or _good(bias, f32, (E,)))):
        _refuse(logits=(logits, (bf16, f32), None), ids=(ids, (torch.int32,), Tk), weights=(weights, (f32,), Tk), bias=(bias, (f32,), (E,)))
    st = (_lib or load()).dg_moe_route(logits.data_ptr(), 1 if kind is f32 else 0, None if bias is None else bias.data_ptr(), ids.data_ptr(),
                                       weights.data_ptr(), T, E, k, _choice(SCORES, scoring, "scoring"), 1 if renormalize else 0, scale,
                                       _stream(stream))
    if st:
        raise DGError(st, "dg_moe_route")
    return ids, weights


def dg_moe_route_backward(logits, ids, dweights, dlogits, scoring="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits [T,E] (the logits' type) from dweights fp32 [T,k], for the ids that dg_moe_route gave."""
    torch = _torch_module or _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    T, E = logits.shape
    k = ids.shape[1]
    kind = logits.dtype
    Tk = (T, k)
    if not ((kind is f32 or kind is bf16) and logits.is_cuda and logits.is_contiguous() and ids.dtype is torch.int32 and ids.shape == Tk
            and ids.is_cuda and ids.is_contiguous() and dweights.dtype is f32 and dweights.shape == Tk and dweights.is_cuda
            and dweights.is_contiguous() and dlogits.dtype is kind and dlogits.shape == (T, E) and dlogits.is_cuda
            and dlogits.is_contiguous()):
        _refuse(logits=(logits, (bf16, f32), None), ids=(ids, (torch.int32,), Tk), dweights=(dweights, (f32,), Tk),
                dlogits=(dlogits, (kind,), (T, E)))
    st = (_lib or load()).dg_moe_route_backward(logits.data_ptr(), 1 if kind is f32 else 0, ids.data_ptr(), dweights.data_ptr(),
                                                dlogits.data_ptr(), T, E, k, _choice(SCORES, scoring, "scoring"),
                                                1 if renormalize else 0, scale, _stream(stream))
    if st:
        raise DGError(st, "dg_moe_route_backward")
    return dlogits


def moe_layer_workspace(T: int, k: int, E: int, H: int, I: int, device=None):
    """A workspace for dg_moe_layer at these sizes, ready for its first call."""
    size = load().dg_moe_layer_workspace(T, k, E, H, I)
    if size < 0:
        raise DGError(2, "dg_moe_layer_workspace")
    return _workspace(size, _MOE_LAYER_ZEROED, device)


def dg_moe_layer(x, ids, weights, W13, s13, W2, s2, out, workspace, act="silu", residual=None, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens:
    out[t] = residual[t] + sum_j weights[t,j] W2[e] . Q(act(g) * u), (g; u) = W13[e] . Q(x[t]), e = ids[t,j];
    x, out, residual bf16 [T,H], ids int32 [T,k] (outside [0,E): no expert), weights fp32 [T,k], W13 e4m3
    [E,2I,H] (gate rows, then up rows), W2 e4m3 [E,H,I], each with fp32 scales per 128x128 block."""
    torch = _torch_module or _torch()
    bf16, f32, e4m3 = torch.bfloat16, torch.float32, (torch.float8_e4m3fn, torch.uint8)
    TH = T, H = x.shape
    k = ids.shape[1]
    E, I2, _ = W13.shape
    I = I2 // 2
    Tk = (T, k)
    if not (W13.dtype in e4m3 and W2.dtype in e4m3 and x.dtype is bf16 and ids.dtype is torch.int32 and weights.dtype is f32
            and out.dtype is bf16 and s13.dtype is f32 and s2.dtype is f32
            and W13.shape == (E, 2 * I, H) and W2.shape == (E, H, I) and s13.shape == (E, I2 // 128, H // 128)
            and s2.shape == (E, H // 128, I // 128) and ids.shape == Tk and weights.shape == Tk and out.shape == TH
            and x.is_cuda and x.is_contiguous() and ids.is_cuda and ids.is_contiguous() and weights.is_cuda and weights.is_contiguous()
            and W13.is_cuda and W13.is_contiguous() and W2.is_cuda and W2.is_contiguous() and s13.is_cuda and s13.is_contiguous()
            and s2.is_cuda and s2.is_contiguous() and out.is_cuda and out.is_contiguous()
            and (residual is None or _good(residual, bf16, TH))):
        _refuse(x=(x, (bf16,), None), ids=(ids, (torch.int32,), Tk), weights=(weights, (f32,), Tk), W13=(W13, e4m3, (E, 2 * I, H)),
                W2=(W2, e4m3, (E, H, I)), s13=(s13, (f32,), (E, I2 // 128, H // 128)), s2=(s2, (f32,), (E, H // 128, I // 128)),
                out=(out, (bf16,), TH), residual=(residual, (bf16,), TH))
    ws, size = _bytes(workspace, "workspace")
    st = (_lib or load()).dg_moe_layer(x.data_ptr(), ids.data_ptr(), weights.data_ptr(), W13.data_ptr(), s13.data_ptr(), W2.data_ptr(),
                                       s2.data_ptr(), None if residual is None else residual.data_ptr(), out.data_ptr(), ws, size,
                                       T, k, E, H, I, _choice(ACTIVATIONS, act, "act"), _stream(stream))
    if st:
        raise DGError(st, "dg_moe_layer")
    return out


def dg_device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) any device-side timeout status."""
    return load().dg_device_status(_stream(stream))


def dg_status_string(status: int) -> str:
    return load().dg_status_string(int(status)).decode()


# Tuning knobs (include/dg_tuning.h): overrides of the automatic tile-shape choice, for sweeps and for
# tests that must reach one kernel specialisation. -1 (or None) is the automatic choice.
TUNE_KNOBS = {"bn": 0, "pair": 1, "split": 2, "swap": 3, "group_m": 4, "pdl": 5}


def dg_tuning_set(knob, value) -> None:
    k = TUNE_KNOBS[knob] if isinstance(knob, str) else int(knob)
    _check(load().dg_tuning_set(k, -1 if value is None else int(value)), "dg_tuning_set")


def dg_tuning_get(knob) -> int:
    return load().dg_tuning_get(TUNE_KNOBS[knob] if isinstance(knob, str) else int(knob))


def dg_tuning_reset() -> None:
    load().dg_tuning_reset()


@contextlib.contextmanager
def tuning(**knobs):
    """Set tuning knobs (bn=, pair=, split=, swap=, group_m=, pdl=) for the duration of a ``with`` block;
    every knob returns to the automatic choice afterwards."""
    try:
        for k, v in knobs.items():
            dg_tuning_set(k, v)
        yield
    finally:
        dg_tuning_reset()


def dg_testing_arm_wait_timeout(wait_limit_ns: int) -> None:
    """Test hook: the next launch of the main kernel bounds its waits by ``wait_limit_ns`` and leaves its
    first pipeline stage unfilled, so that a wait runs out and the kernel reports DG_DEVICE_TIMEOUT."""
    _check(load().dg_testing_arm_wait_timeout(int(wait_limit_ns)), "dg_testing_arm_wait_timeout")


# What an armed launch leaves out (include/dg_tuning.h).
FAULTS = {"first_fill": 1, "residual": 2, "token_scales": 3, "grid_barrier": 4}


def dg_testing_arm_fault(fault, wait_limit_ns: int) -> None:
    """Test hook: the next launch bounds its waits by ``wait_limit_ns`` and leaves out what ``fault`` names (a
    name of FAULTS or its number), so that the wait for it runs out and the kernel reports DG_DEVICE_TIMEOUT."""
    _check(load().dg_testing_arm_fault(FAULTS[fault] if isinstance(fault, str) else int(fault), int(wait_limit_ns)), "dg_testing_arm_fault")
