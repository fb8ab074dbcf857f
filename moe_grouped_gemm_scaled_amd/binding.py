"""ctypes binding of libdg.so (C ABI in include/dg.h).

Argument marshalling only: the functions check that tensors have the dtype,
device, contiguity and shape the C ABI documents, then pass raw device
pointers, sizes and the current HIP stream.  Every step of the computation
runs in the library's HIP kernels.  There is no fallback: if libdg.so is
missing, loading raises.

E4M3 tensors may be torch.uint8 or torch.float8_e4m3fn; bf16 tensors are
torch.bfloat16; scales torch.float32; index tensors torch.int32.
"""
from __future__ import annotations

import ctypes as ct
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK = 0
_STATUS = {0: "DG_OK", -1: "DG_ERR_NULL", -2: "DG_ERR_SHAPE", -3: "DG_ERR_ALIGN", -4: "DG_ERR_ARG",
           -5: "DG_ERR_UNSUPPORTED", -6: "DG_ERR_HIP", -7: "DG_ERR_SCRATCH"}

_P = ct.c_void_p

EXPORTS = {
    # name: (restype, argtypes)
    "dg_fp8_gemm_nt": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                  ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_nt_ws": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                     ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p, ct.c_size_t,
                                     ct.c_void_p]),
    "dg_fp8_gemm_nt_ue8m0_ws": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p,
                                           ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p,
                                           ct.c_size_t, ct.c_void_p]),
    "dg_get_workspace_size": (ct.c_int64, [ct.c_int, ct.c_int, ct.c_int]),
    "dg_fp8_gemm_nt_noalloc": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p,
                                          ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_contiguous": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                       ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int,
                                                       ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_masked": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                   ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int,
                                                   ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_quantize_e4m3_1x128": (ct.c_int, [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p, ct.c_void_p,
                                          ct.c_int, ct.c_void_p]),
    "dg_quantize_e4m3_128x128": (ct.c_int, [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p, ct.c_void_p,
                                            ct.c_void_p]),
    "dg_fp8_gemm_nt_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                        ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                             ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int,
                                                             ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_masked_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                         ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int,
                                                         ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_quantize_e4m3_1x128_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p,
                                                ct.c_void_p, ct.c_int, ct.c_void_p]),
    "dg_quantize_e4m3_128x128_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p,
                                                  ct.c_void_p, ct.c_void_p]),
    "dg_fp8_gemm_nn": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                  ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_tn": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                  ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_tt": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                  ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_k_grouped_fp8_gemm_tn_contiguous": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                       ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int,
                                                       ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_nn_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                        ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_tn_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                        ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_tt_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                        ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_k_grouped_fp8_gemm_tn_contiguous_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                             ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_int,
                                                             ct.c_int, ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_fp8_gemm_nt_ue8m0_packed": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_void_p,
                                               ct.c_void_p, ct.c_void_p, ct.c_int, ct.c_int, ct.c_int,
                                               ct.c_void_p, ct.c_size_t, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                                    ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                                    ct.c_void_p, ct.c_int, ct.c_int, ct.c_int,
                                                                    ct.c_int, ct.c_void_p]),
    "dg_m_grouped_fp8_gemm_nt_masked_ue8m0_packed": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                                ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                                                ct.c_void_p, ct.c_int, ct.c_int, ct.c_int,
                                                                ct.c_int, ct.c_int, ct.c_void_p]),
    "dg_pack_sf_ue8m0": (ct.c_int, [ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_void_p, ct.c_void_p]),
    "dg_fp8_mqa_logits": (ct.c_int, [ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p, ct.c_void_p,
                                     ct.c_void_p, ct.c_int, ct.c_void_p, ct.c_int, ct.c_int, ct.c_int, ct.c_int,
                                     ct.c_void_p]),
    "dg_get_mk_alignment_for_contiguous_layout": (ct.c_int, []),
    **{name: (ct.c_int, [_P, ct.c_int, ct.c_int64, _P, ct.c_int, _P, ct.c_int, ct.c_float, _P, _P, _P, _P, ct.c_int,
                         ct.c_int, ct.c_int, _P])
       for name in ("dg_rmsnorm_quantize_e4m3_1x128", "dg_rmsnorm_quantize_e4m3_1x128_ue8m0",
                    "dg_rmsnorm_quantize_e4m3_1x128_ue8m0_packed")},
    "dg_rmsnorm_backward": (ct.c_int, [_P, ct.c_int, _P, ct.c_int, _P, ct.c_int, ct.c_float, _P, _P, _P, ct.c_int,
                                       ct.c_int, _P, ct.c_size_t, _P]),
    "dg_get_rmsnorm_backward_workspace_size": (ct.c_int64, [ct.c_int, ct.c_int]),
    **{name: (ct.c_int, [_P, _P, ct.c_int, _P, _P, ct.c_int, _P, _P, _P, _P, ct.c_int, ct.c_int, ct.c_int, ct.c_int,
                         _P, ct.c_size_t, _P])
       for name in ("dg_fp8_gated_gemm_nt", "dg_fp8_gated_gemm_nt_ue8m0_packed")},
    "dg_get_gated_workspace_size": (ct.c_int64, [ct.c_int, ct.c_int, ct.c_int]),
    **{name: (ct.c_int, [_P, _P, _P, _P, ct.c_int, _P, _P, _P, _P, _P, ct.c_int, ct.c_int, ct.c_int, ct.c_int, _P])
       for name in ("dg_m_grouped_fp8_gated_gemm_nt_contiguous",
                    "dg_m_grouped_fp8_gated_gemm_nt_contiguous_ue8m0_packed")},
    **{name: (ct.c_int, [_P, _P, _P, _P, ct.c_int, _P, _P, _P, _P, _P, ct.c_int, ct.c_int, ct.c_int, ct.c_int,
                         ct.c_int, _P])
       for name in ("dg_m_grouped_fp8_gated_gemm_nt_masked", "dg_m_grouped_fp8_gated_gemm_nt_masked_ue8m0_packed")},
    **{name: (ct.c_int, [_P, _P, ct.c_int, _P, _P, _P, _P, ct.c_int, _P, _P, _P, _P, ct.c_int, ct.c_int, _P])
       for name in ("dg_gated_backward_quantize_e4m3", "dg_gated_backward_quantize_e4m3_ue8m0")},
    "dg_set_mk_alignment_for_contiguous_layout": (ct.c_int, [ct.c_int]),
    "dg_get_sf_aligned_size": (ct.c_int, [ct.c_int]),
    "dg_set_num_cus": (ct.c_int, [ct.c_int]),
    "dg_get_num_cus": (ct.c_int, []),
    "dg_set_kernel_family": (ct.c_int, [ct.c_char_p]),
    "dg_get_kernel_family": (ct.c_char_p, []),
    "dg_status_string": (ct.c_char_p, [ct.c_int]),
    "dg_last_config": (ct.c_char_p, []),
}

_lib = None
_lock = threading.Lock()


class DGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)} ({lib().dg_status_string(status).decode()})")


def lib() -> ct.CDLL:
    """The loaded libdg.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise ImportError(f"{LIB_PATH} is missing: build it with "
                                      "`python -m moe_grouped_gemm_scaled_amd.build`")
                l = ct.CDLL(LIB_PATH)
                for name, (res, args) in EXPORTS.items():
                    f = getattr(l, name)
                    f.restype = res
                    f.argtypes = args
                _lib = l
    return _lib


def _check(status: int, where: str):
    if status != DG_OK:
        raise DGError(status, where)


def _stream(t: torch.Tensor):
    return ct.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


_FP8 = (torch.uint8, torch.float8_e4m3fn)


def _ptr(t, dtypes, name, shape=None):
    if t is None:
        return None
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ct.c_void_p(t.data_ptr())


def ceil_div(a: int, b: int) -> int:
    return (a + b - 1) // b


def _name(base: str, ue8m0: bool) -> str:
    return base + "_ue8m0" if ue8m0 else base


def get_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of split-K scratch dg_fp8_gemm_nt_ws needs for M x N x K on the current device (0: no split)."""
    v = lib().dg_get_workspace_size(int(M), int(N), int(K))
    if v < 0:
        raise DGError(int(v), "dg_get_workspace_size")
    return int(v)


def get_workspace(M: int, N: int, K: int, device=None):
    """A zero-filled uint8 device tensor of get_workspace_size(M, N, K) bytes (None when the problem does
    not split K).  It may serve any number of fp8_gemm_nt calls in stream order; calls that can run at
    the same time (other streams, graphs replayed concurrently) each need their own."""
    n = get_workspace_size(M, N, K)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def fp8_gemm_nt(a, sfa, b, sfb, d, c=None, ue8m0=False, workspace="auto"):
    """D = C + A . B^T.  a[M,K], sfa[K/128, ld_sfa], b[N,K], sfb[ceil(N/128), K/128], d/c[M,N] bf16.
    ue8m0: every scale is a power of two (dg_fp8_gemm_nt_ue8m0[_ws]).
    workspace: a zeroed uint8 device tensor from get_workspace() (dg_fp8_gemm_nt_ws); None runs without
    split-K (dg_fp8_gemm_nt); "auto" takes a fresh zeroed one from torch's allocator for this call."""
    M, K = a.shape
    N = b.shape[0]
    if sfa.dim() != 2 or sfa.shape[0] != K // 128:
        raise ValueError(f"sfa: shape {tuple(sfa.shape)}, expected [K/128={K // 128}, ld_sfa]")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace {workspace!r}")
        workspace = get_workspace(M, N, K, d.device)
    args = (_ptr(a, _FP8, "a", (M, K)), _ptr(sfa, torch.float32, "sfa"), int(sfa.shape[1]),
            _ptr(b, _FP8, "b", (N, K)), _ptr(sfb, torch.float32, "sfb", (ceil_div(N, 128), K // 128)),
            _ptr(c, torch.bfloat16, "c", (M, N)), _ptr(d, torch.bfloat16, "d", (M, N)), M, N, K)
    if workspace is None:
        name = _name("dg_fp8_gemm_nt", ue8m0)
        _check(getattr(lib(), name)(*args, _stream(d)), name)
    else:
        name = "dg_fp8_gemm_nt_ue8m0_ws" if ue8m0 else "dg_fp8_gemm_nt_ws"
        ws = _ptr(workspace, torch.uint8, "workspace")
        _check(getattr(lib(), name)(*args, ws, int(workspace.numel()), _stream(d)), name)
    return d


def fp8_gemm_nt_noalloc(a, sfa, b, sfb, d, c=None):
    """D = C + A . B^T through dg_fp8_gemm_nt_noalloc: split-K scratch from the library's own device array,
    nothing allocated (not even by torch); calls that may overlap on one GPU race.  Arguments as for
    fp8_gemm_nt."""
    M, K = a.shape
    N = b.shape[0]
    if sfa.dim() != 2 or sfa.shape[0] != K // 128:
        raise ValueError(f"sfa: shape {tuple(sfa.shape)}, expected [K/128={K // 128}, ld_sfa]")
    args = (_ptr(a, _FP8, "a", (M, K)), _ptr(sfa, torch.float32, "sfa"), int(sfa.shape[1]),
            _ptr(b, _FP8, "b", (N, K)), _ptr(sfb, torch.float32, "sfb", (ceil_div(N, 128), K // 128)),
            _ptr(c, torch.bfloat16, "c", (M, N)), _ptr(d, torch.bfloat16, "d", (M, N)), M, N, K, _stream(d))
    _check(lib().dg_fp8_gemm_nt_noalloc(*args), "dg_fp8_gemm_nt_noalloc")
    return d


def fp8_gemm(layout, a, sfa, b, sfb, d, c=None, ue8m0=False):
    """D = C + A @ B in one of the layouts "nt", "nn", "tn", "tt" (dg_fp8_gemm_<layout>).
    The first letter is A's storage: "n" a[M,K], "t" a[K,M]; the second B's: "t" b[N,K], "n" b[K,N].
    Scales as for fp8_gemm_nt: sfa[K/128, ld_sfa], sfb[ceil(N/128), K/128]; d/c[M,N] bf16."""
    if layout not in ("nt", "nn", "tn", "tt"):
        raise ValueError(f"layout {layout!r}")
    M, N = d.shape
    K = a.shape[1] if layout[0] == "n" else a.shape[0]
    a_shape = (M, K) if layout[0] == "n" else (K, M)
    b_shape = (N, K) if layout[1] == "t" else (K, N)
    if sfa.dim() != 2 or sfa.shape[0] != K // 128:
        raise ValueError(f"sfa: shape {tuple(sfa.shape)}, expected [K/128={K // 128}, ld_sfa]")
    args = (_ptr(a, _FP8, "a", a_shape), _ptr(sfa, torch.float32, "sfa"), int(sfa.shape[1]),
            _ptr(b, _FP8, "b", b_shape), _ptr(sfb, torch.float32, "sfb", (ceil_div(N, 128), K // 128)),
            _ptr(c, torch.bfloat16, "c", (M, N)), _ptr(d, torch.bfloat16, "d", (M, N)), M, N, K, _stream(d))
    name = _name("dg_fp8_gemm_" + layout, ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return d


def k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, ks, d, c=None, ue8m0=False):
    """K-grouped TN contiguous GEMM (dg_k_grouped_fp8_gemm_tn_contiguous): a[K,M], b[K,N] E4M3,
    sfa[K/128,M], sfb[K/128,N] fp32, ks[G] int32 device tensor of group sizes (multiples of 128),
    d (and c, optional, may be d) fp32 [G,M,N]:  D[g] = C[g] + A_g^T B_g."""
    K, M = a.shape
    N = b.shape[1]
    G = ks.shape[0]
    args = (_ptr(a, _FP8, "a", (K, M)), _ptr(sfa, torch.float32, "sfa", (K // 128, M)),
            _ptr(b, _FP8, "b", (K, N)), _ptr(sfb, torch.float32, "sfb", (K // 128, N)),
            _ptr(ks, torch.int32, "ks", (G,)), _ptr(c, torch.float32, "c", (G, M, N)),
            _ptr(d, torch.float32, "d", (G, M, N)), M, N, K, G, _stream(d))
    name = _name("dg_k_grouped_fp8_gemm_tn_contiguous", ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return d


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices, c=None, ue8m0=False):
    """a[M_total,K], sfa[K/128, M_total], b[G,N,K], sfb[G, ceil(N/128), K/128], d/c[M_total,N], m_indices[M_total]."""
    M_total, K = a.shape
    G, N, _ = b.shape
    args = (_ptr(a, _FP8, "a", (M_total, K)), _ptr(sfa, torch.float32, "sfa", (K // 128, M_total)),
            _ptr(b, _FP8, "b", (G, N, K)), _ptr(sfb, torch.float32, "sfb", (G, ceil_div(N, 128), K // 128)),
            _ptr(c, torch.bfloat16, "c", (M_total, N)), _ptr(d, torch.bfloat16, "d", (M_total, N)),
            _ptr(m_indices, torch.int32, "m_indices", (M_total,)), M_total, N, K, G, _stream(d))
    name = _name("dg_m_grouped_fp8_gemm_nt_contiguous", ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return d


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, expected_m=0, c=None, ue8m0=False):
    """a[G,M_cap,K], sfa[G, K/128, round_up(M_cap,4)], b[G,N,K], sfb[G, ceil(N/128), K/128], d/c[G,M_cap,N]."""
    G, M_cap, K = a.shape
    N = b.shape[1]
    ld = (M_cap + 3) // 4 * 4
    args = (_ptr(a, _FP8, "a", (G, M_cap, K)), _ptr(sfa, torch.float32, "sfa", (G, K // 128, ld)),
            _ptr(b, _FP8, "b", (G, N, K)), _ptr(sfb, torch.float32, "sfb", (G, ceil_div(N, 128), K // 128)),
            _ptr(c, torch.bfloat16, "c", (G, M_cap, N)), _ptr(d, torch.bfloat16, "d", (G, M_cap, N)),
            _ptr(masked_m, torch.int32, "masked_m", (G,)), G, M_cap, N, K, int(expected_m), _stream(d))
    name = _name("dg_m_grouped_fp8_gemm_nt_masked", ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return d


def quantize_e4m3_1x128(x, q=None, sf=None, ld_sf=None, ue8m0=False):
    """x[groups, rows, K] or [rows, K] fp32 -> (q uint8, sf[groups, K/128, ld_sf] or [K/128, ld_sf]).
    ue8m0: power-of-two scales (dg_quantize_e4m3_1x128_ue8m0)."""
    squeeze = x.dim() == 2
    groups, rows, K = (1,) + tuple(x.shape) if squeeze else tuple(x.shape)
    ld = (rows + 3) // 4 * 4 if ld_sf is None else int(ld_sf)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.zeros((K // 128, ld) if squeeze else (groups, K // 128, ld), dtype=torch.float32, device=x.device)
    _ptr(sf, torch.float32, "sf", (K // 128, ld) if squeeze else (groups, K // 128, ld))
    args = (_ptr(x, torch.float32, "x"), groups, rows, K, _ptr(q, _FP8, "q", tuple(x.shape)),
            ct.c_void_p(sf.data_ptr()), ld, _stream(x))
    name = _name("dg_quantize_e4m3_1x128", ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return q, sf


def quantize_e4m3_128x128(x, q=None, sf=None, ue8m0=False):
    """x[groups, rows, K] or [rows, K] fp32 -> (q uint8, sf[groups, ceil(rows/128), K/128]).
    ue8m0: power-of-two scales (dg_quantize_e4m3_128x128_ue8m0)."""
    squeeze = x.dim() == 2
    groups, rows, K = (1,) + tuple(x.shape) if squeeze else tuple(x.shape)
    shape_sf = (ceil_div(rows, 128), K // 128) if squeeze else (groups, ceil_div(rows, 128), K // 128)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(shape_sf, dtype=torch.float32, device=x.device)
    args = (_ptr(x, torch.float32, "x"), groups, rows, K, _ptr(q, _FP8, "q", tuple(x.shape)),
            _ptr(sf, torch.float32, "sf", shape_sf), _stream(x))
    name = _name("dg_quantize_e4m3_128x128", ue8m0)
    _check(getattr(lib(), name)(*args), name)
    return q, sf


def pack_sf_ue8m0(sf, k_axis, out=None):
    """Packs power-of-two fp32 scales four per 32-bit word along the K-block axis `k_axis`
    (dg_pack_sf_ue8m0): byte j of word q holds the exponent field of K block 4q + j.  sfa [.., K/128, ld]
    takes k_axis=-2, sfb [.., ceil(N/128), K/128] k_axis=-1.  Returns int32 words of sf's shape with
    ceil(K/512) along k_axis."""
    shape = tuple(sf.shape)
    ax = k_axis % len(shape)
    outer = 1
    for v in shape[:ax]:
        outer *= v
    inner = 1
    for v in shape[ax + 1:]:
        inner *= v
    kblocks = shape[ax]
    out_shape = shape[:ax] + (ceil_div(kblocks, 4),) + shape[ax + 1:]
    if out is None:
        out = torch.empty(out_shape, dtype=torch.int32, device=sf.device)
    _check(lib().dg_pack_sf_ue8m0(_ptr(sf, torch.float32, "sf"), outer, kblocks, inner,
                                  _ptr(out, torch.int32, "out", out_shape), _stream(sf)), "dg_pack_sf_ue8m0")
    return out


def fp8_gemm_nt_ue8m0_packed(a, sfa, b, sfb, d, c=None, workspace="auto"):
    """D = C + A . B^T on packed power-of-two scales (dg_fp8_gemm_nt_ue8m0_packed): sfa int32
    [ceil(K/512), ld_sfa], sfb int32 [ceil(N/128), ceil(K/512)] as pack_sf_ue8m0 writes them; the other
    arguments as for fp8_gemm_nt (workspace None: no split-K)."""
    M, K = a.shape
    N = b.shape[0]
    nkw = ceil_div(K // 128, 4)
    if sfa.dim() != 2 or sfa.shape[0] != nkw:
        raise ValueError(f"sfa: shape {tuple(sfa.shape)}, expected [ceil(K/512)={nkw}, ld_sfa]")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace {workspace!r}")
        workspace = get_workspace(M, N, K, d.device)
    ws = _ptr(workspace, torch.uint8, "workspace")
    args = (_ptr(a, _FP8, "a", (M, K)), _ptr(sfa, torch.int32, "sfa"), int(sfa.shape[1]),
            _ptr(b, _FP8, "b", (N, K)), _ptr(sfb, torch.int32, "sfb", (ceil_div(N, 128), nkw)),
            _ptr(c, torch.bfloat16, "c", (M, N)), _ptr(d, torch.bfloat16, "d", (M, N)), M, N, K,
            ws, int(workspace.numel()) if workspace is not None else 0, _stream(d))
    _check(lib().dg_fp8_gemm_nt_ue8m0_packed(*args), "dg_fp8_gemm_nt_ue8m0_packed")
    return d


def m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed(a, sfa, b, sfb, d, m_indices, c=None):
    """Contiguous grouped GEMM on packed power-of-two scales: sfa int32 [ceil(K/512), M_total], sfb int32
    [G, ceil(N/128), ceil(K/512)]; the rest as m_grouped_fp8_gemm_nt_contiguous."""
    M_total, K = a.shape
    G, N, _ = b.shape
    nkw = ceil_div(K // 128, 4)
    args = (_ptr(a, _FP8, "a", (M_total, K)), _ptr(sfa, torch.int32, "sfa", (nkw, M_total)),
            _ptr(b, _FP8, "b", (G, N, K)), _ptr(sfb, torch.int32, "sfb", (G, ceil_div(N, 128), nkw)),
            _ptr(c, torch.bfloat16, "c", (M_total, N)), _ptr(d, torch.bfloat16, "d", (M_total, N)),
            _ptr(m_indices, torch.int32, "m_indices", (M_total,)), M_total, N, K, G, _stream(d))
    _check(lib().dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed(*args),
           "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0_packed")
    return d


def m_grouped_fp8_gemm_nt_masked_ue8m0_packed(a, sfa, b, sfb, d, masked_m, expected_m=0, c=None):
    """Masked grouped GEMM on packed power-of-two scales: sfa int32 [G, ceil(K/512), round_up(M_cap,4)],
    sfb int32 [G, ceil(N/128), ceil(K/512)]; the rest as m_grouped_fp8_gemm_nt_masked."""
    G, M_cap, K = a.shape
    N = b.shape[1]
    ld = (M_cap + 3) // 4 * 4
    nkw = ceil_div(K // 128, 4)
    args = (_ptr(a, _FP8, "a", (G, M_cap, K)), _ptr(sfa, torch.int32, "sfa", (G, nkw, ld)),
            _ptr(b, _FP8, "b", (G, N, K)), _ptr(sfb, torch.int32, "sfb", (G, ceil_div(N, 128), nkw)),
            _ptr(c, torch.bfloat16, "c", (G, M_cap, N)), _ptr(d, torch.bfloat16, "d", (G, M_cap, N)),
            _ptr(masked_m, torch.int32, "masked_m", (G,)), G, M_cap, N, K, int(expected_m), _stream(d))
    _check(lib().dg_m_grouped_fp8_gemm_nt_masked_ue8m0_packed(*args), "dg_m_grouped_fp8_gemm_nt_masked_ue8m0_packed")
    return d


def fp8_mqa_logits(q, kv, kv_scale, weights, k_start, k_end, clean_logits=True, logits=None):
    """FP8 MQA logits (dg_fp8_mqa_logits).  q[S, H, D], kv[S_kv, D] E4M3, kv_scale[S_kv] fp32,
    weights[S, H] fp32, k_start/k_end[S] int32 -> logits[S, S_kv] fp32 (allocated when None; when
    clean_logits is false, positions outside a row's range keep what `logits` held)."""
    S, H, D = tuple(q.shape)
    S_kv = kv.shape[0]
    if logits is None:
        logits = torch.empty((S, S_kv), dtype=torch.float32, device=q.device)
    args = (_ptr(q, _FP8, "q"), _ptr(kv, _FP8, "kv", (S_kv, D)), _ptr(kv_scale, torch.float32, "kv_scale", (S_kv,)),
            _ptr(weights, torch.float32, "weights", (S, H)), _ptr(k_start, torch.int32, "k_start", (S,)),
            _ptr(k_end, torch.int32, "k_end", (S,)), int(bool(clean_logits)),
            _ptr(logits, torch.float32, "logits", (S, S_kv)), S, H, D, S_kv, _stream(q))
    _check(lib().dg_fp8_mqa_logits(*args), "dg_fp8_mqa_logits")
    return logits


# ---------------------------------------------------------------- the feed-forward layer

_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_ACTS = {"silu": 0, "gelu": 1}
_SUFFIX = {"fp32": "", "ue8m0": "_ue8m0", "ue8m0_packed": "_ue8m0_packed"}

# Type sets of arguments, as the bits that the native checks use.
_BF16, _F32, _REAL, _E4M3, _I32 = 1, 2, 3, 12, 16
_BIT_TYPES = {_BF16: torch.bfloat16, _F32: torch.float32, _REAL: (torch.bfloat16, torch.float32), _E4M3: _FP8,
              _I32: torch.int32}

# the current stream's handle without making a torch.cuda.Stream object (2.7 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

try:
    from ._args import addresses as _native_addresses   # csrc/py_args.cpp: the checks of _raw, natively
except ImportError:                                     # not built: the same checks in Python
    def _native_addresses(*_):
        return None


def _raw(t, dtype, shape, name):
    """The address of a dense device tensor of this type (or one of a tuple) and shape; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _device(t, name):
    """The device of a call's tensors, which has to be the current device (kernels run there)."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name}: must be a device tensor")
    if index != torch.cuda.current_device():
        raise ValueError(f"{name}: on device {index}, but the current device is {torch.cuda.current_device()}")
    return index


def _pointers(index, names, *specs):
    """Addresses of the tensors in specs = t0, types0, shape0, t1, .. (None for None), all checked."""
    got = _native_addresses(index, *specs)
    if got is None:
        got = []
        for name, t, bits, shape in zip(names, specs[0::3], specs[1::3], specs[2::3]):
            got.append(_raw(t, _BIT_TYPES[bits], shape, name))
            if t is not None and t.get_device() != index:
                raise ValueError(f"{name}: on device {t.get_device()}, other arguments on device {index}")
    return got


def _type_of(t, name):
    try:
        return _TYPES[t.dtype]
    except (KeyError, AttributeError):
        raise TypeError(f"{name}: {getattr(t, 'dtype', t)}, expected a tensor of torch.bfloat16 or torch.float32") from None


def _act_of(act):
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act {act!r}, expected one of {tuple(_ACTS)}") from None


def _out(t, shape, dtype, device, zero=False):
    """An output argument: a tensor as given, a new one for True, None otherwise."""
    if t is True:
        return torch.zeros(shape, dtype=dtype, device=device) if zero else torch.empty(shape, dtype=dtype, device=device)
    return None if t is False else t


_functions = {}


def _call(name, *args):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    status = f(*args)
    if status != DG_OK:
        raise DGError(status, name)


def _sf_rows(packed, kblocks):
    return (kblocks + 3) // 4 if packed else kblocks


_NORM_NAMES = ("residual", "weight", "residual_out", "y", "q", "sf")


def rmsnorm_quantize_e4m3_1x128(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, q=None, sf=None,
                                ld_sf=None, scales="fp32"):
    """h = x + residual, RMS norm of h times weight, 1x128 E4M3 quantisation, in one pass
    (dg_rmsnorm_quantize_e4m3_1x128[_ue8m0[_packed]]).

    x[rows, K] bf16 or fp32 (rows may be strided, columns dense), weight[K] bf16 or fp32; residual[rows, K] bf16 or
    fp32, with residual_out (allocated when None; may be the residual itself) receiving h; y: a bf16 [rows, K] tensor
    to fill, or True for a new one; scales "fp32" or "ue8m0" (sf[K/128, ld_sf] fp32) or "ue8m0_packed"
    (sf[ceil(K/512), ld_sf] int32).  q=False leaves the quantised output out (y is needed then).
    Returns (q, sf, residual_out, y), None where not asked for."""
    suffix = _SUFFIX.get(scales)
    if suffix is None:
        raise ValueError(f"scales {scales!r}, expected one of {tuple(_SUFFIX)}")
    if x.dim() != 2:
        raise ValueError("x: must have two dimensions, [rows, K]")
    shape = x.shape
    rows, K = shape
    pitch, column = x.stride()
    if column != 1 and K > 1:
        raise ValueError("x: columns must be dense")
    index = _device(x, "x")
    res_type = 0
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
    else:
        res_type = _type_of(residual, "residual")
        if residual_out is None:
            residual_out = torch.empty_like(residual)
    if y is True:
        y = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    packed = scales == "ue8m0_packed"
    ld, sf_shape = 0, ()
    if q is False:
        q = sf = None
    else:
        ld = (sf.shape[-1] if sf is not None else (rows + 3) // 4 * 4) if ld_sf is None else int(ld_sf)
        sf_shape = (_sf_rows(packed, K // 128), ld)
        if q is None:
            q = torch.empty(shape, dtype=torch.uint8, device=x.device)
        if sf is None:
            sf = torch.zeros(sf_shape, dtype=torch.int32 if packed else torch.float32, device=x.device)
    res_bits = _F32 if res_type else _BF16
    p = _pointers(index, _NORM_NAMES, residual, res_bits, shape, weight, _REAL, (K,), residual_out, res_bits, shape,
                  y, _BF16, shape, q, _E4M3, shape, sf, _I32 if packed else _F32, sf_shape)
    _call("dg_rmsnorm_quantize_e4m3_1x128" + suffix, x.data_ptr(), _type_of(x, "x"), pitch if rows > 1 else K, p[0],
          res_type, p[1], _type_of(weight, "weight"), eps, p[2], p[3], p[4], p[5], ld, rows, K, _raw_stream(index))
    return q, sf, residual_out, y


def get_rmsnorm_backward_workspace_size(rows: int, K: int) -> int:
    """Bytes of scratch rmsnorm_backward needs on the current device (of any content)."""
    v = lib().dg_get_rmsnorm_backward_workspace_size(int(rows), int(K))
    if v < 0:
        raise DGError(int(v), "dg_get_rmsnorm_backward_workspace_size")
    return int(v)


_NORM_BWD_NAMES = ("dy", "h", "weight", "dres", "dx", "dw")


def rmsnorm_backward(dy, h, weight, eps=1e-6, dres=None, dx=None, dw=None, workspace="auto"):
    """Gradient of the RMS norm (dg_rmsnorm_backward): dy[rows, K] bf16 or fp32, h[rows, K] the norm's input as stored
    (bf16 or fp32), dres[rows, K] of h's type the gradient arriving at h itself (or None); returns (dx of h's type,
    dw[K] fp32).  dx may be dres or h.  workspace: a uint8 device tensor of get_rmsnorm_backward_workspace_size bytes,
    or "auto"."""
    shape = h.shape
    if len(shape) != 2:
        raise ValueError(f"h: shape {tuple(shape)}, expected [rows, K]")
    rows, K = shape
    if isinstance(workspace, str) and workspace != "auto":
        raise ValueError(f"workspace {workspace!r}")
    index = _device(h, "h")
    h_type = _type_of(h, "h")
    if isinstance(workspace, str):
        n = get_rmsnorm_backward_workspace_size(rows, K)
        workspace = torch.empty(n, dtype=torch.uint8, device=h.device) if n else None
    if dx is None:
        dx = torch.empty_like(h)
    if dw is None:
        dw = torch.empty(K, dtype=torch.float32, device=h.device)
    bits = _F32 if h_type else _BF16
    p = _pointers(index, _NORM_BWD_NAMES, dy, _REAL, shape, h, bits, shape, weight, _REAL, (K,), dres, bits, shape,
                  dx, bits, shape, dw, _F32, (K,))
    _call("dg_rmsnorm_backward", p[0], _type_of(dy, "dy"), p[1], h_type, p[2], _type_of(weight, "weight"), eps, p[3],
          p[4], p[5], rows, K, *_workspace(workspace, index), _raw_stream(index))
    return dx, dw


def _workspace(t, index):
    """Address and bytes of a workspace argument."""
    if t is None:
        return None, 0
    if t.get_device() != index:
        raise ValueError(f"workspace: on device {t.get_device()}, other arguments on device {index}")
    return _raw(t, torch.uint8, t.shape, "workspace"), t.numel()


def get_gated_workspace_size(M: int, I: int, K: int) -> int:
    """Bytes of scratch (of any content) fp8_gated_gemm_nt uses for a quantised output on the current device (0: none)."""
    v = lib().dg_get_gated_workspace_size(int(M), int(I), int(K))
    if v < 0:
        raise DGError(int(v), "dg_get_gated_workspace_size")
    return int(v)


_GATED_NAMES = ("a", "sfa", "b", "sfb", "gu", "h", "q", "sf")


def _gated_args(a, sfa, b, sfb, act, h, q, sf, gu, lead, G, rows, ld):
    """Arguments that the three layouts of the gated GEMM share, and the outputs: lead = leading dimensions of the
    row tensors, G = leading dimensions of b."""
    index = _device(a, "a")
    I, K = b.shape[-2:]
    packed = sfa.dtype is torch.int32
    sf_bits = _I32 if packed else _F32
    n, blocks = _sf_rows(packed, K // 128), (I + 127) // 128
    if h is None and q is None and sf is None:
        h = True
    partial = len(G) > 0                       # rows without data keep what the buffers hold
    shape_h = (*lead, rows, I)
    shape_gu = (*lead, rows, 2 * I)
    shape_sf = (*lead, _sf_rows(packed, blocks), ld)
    if h is True or q is True or gu is True or (q is not None and sf is None) or sf is True:
        dev = a.device
        h = _out(h, shape_h, torch.bfloat16, dev, partial)
        gu = _out(gu, shape_gu, torch.bfloat16, dev, partial)
        q = _out(q, shape_h, torch.uint8, dev, partial)
        if q is not None and (sf is None or sf is True):
            sf = torch.zeros(shape_sf, dtype=torch.int32 if packed else torch.float32, device=dev)
    if q is None:
        sf = None
    if gu is not None and gu.dim() == len(lead) + 3:
        shape_gu = (*lead, rows, 2, I)
    p = _pointers(index, _GATED_NAMES, a, _E4M3, (*lead, rows, K), sfa, sf_bits, (*lead, n, ld), b, _E4M3, (*G, 2, I, K),
                  sfb, sf_bits, (*G, 2, blocks, n), gu, _BF16, shape_gu, h, _BF16, shape_h, q, _E4M3, shape_h,
                  sf, sf_bits, shape_sf)
    return p, _act_of(act), (h, q, sf, gu), I, K, "_ue8m0_packed" if packed else "", index


def fp8_gated_gemm_nt(a, sfa, b, sfb, act="silu", h=None, q=None, sf=None, gu=None, workspace="auto"):
    """h = act(A Wg^T) * (A Wu^T) in one kernel (dg_fp8_gated_gemm_nt): a[M, K], sfa[K/128, ld], b[2, I, K] (Wg, Wu),
    sfb[2, ceil(I/128), K/128]; int32 sfa and sfb are packed power-of-two scales (dg_fp8_gated_gemm_nt_ue8m0_packed).
    act "silu" or "gelu" (tanh form).  Outputs: a tensor to fill, or True for a new one: h[M, I] bf16 (the default),
    q[M, I] E4M3 with sf[I/128 (packed: ceil(I/512)), ld], gu[M, 2I] bf16 (gate, up).  workspace (used for q of small problems): a
    uint8 device tensor of get_gated_workspace_size(M, I, K) bytes, None for none, or "auto".  Returns (h, q, sf, gu),
    None where not asked for."""
    if a.dim() != 2 or b.dim() != 3 or sfa.dim() != 2:
        raise ValueError("a[M, K], sfa[K/128, ld], b[2, I, K]")
    M = a.shape[0]
    ld = sfa.shape[1]
    p, act_id, ret, I, K, suffix, index = _gated_args(a, sfa, b, sfb, act, h, q, sf, gu, (), (), M, ld)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace {workspace!r}")
        n = get_gated_workspace_size(M, I, K) if ret[1] is not None else 0
        workspace = torch.empty(n, dtype=torch.uint8, device=a.device) if n else None
    _call("dg_fp8_gated_gemm_nt" + suffix, p[0], p[1], ld, p[2], p[3], act_id, p[4], p[5], p[6], p[7], ld, M, I, K,
          *_workspace(workspace, index), _raw_stream(index))
    return ret


def m_grouped_fp8_gated_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, act="silu", h=None, q=None, sf=None, gu=None):
    """The gated GEMM in the contiguous layout: a[M_total, K], sfa[K/128, M_total], b[G, 2, I, K],
    sfb[G, 2, ceil(I/128), K/128], m_indices[M_total] int32; outputs as fp8_gated_gemm_nt (ld = M_total), new ones
    zero on the rows without data."""
    if a.dim() != 2 or b.dim() != 4:
        raise ValueError("a[M_total, K], b[G, 2, I, K]")
    M, G = a.shape[0], b.shape[0]
    p, act_id, ret, I, K, suffix, index = _gated_args(a, sfa, b, sfb, act, h, q, sf, gu, (), (G,), M, M)
    idx = _pointers(index, ("m_indices",), m_indices, _I32, (M,))
    _call("dg_m_grouped_fp8_gated_gemm_nt_contiguous" + suffix, p[0], p[1], p[2], p[3], act_id, p[4], p[5], p[6], p[7],
          idx[0], M, I, K, G, _raw_stream(index))
    return ret


def m_grouped_fp8_gated_gemm_nt_masked(a, sfa, b, sfb, masked_m, expected_m=0, act="silu", h=None, q=None, sf=None,
                                       gu=None):
    """The gated GEMM in the masked layout: a[G, M_cap, K], sfa[G, K/128, round_up(M_cap, 4)], b[G, 2, I, K],
    sfb[G, 2, ceil(I/128), K/128], masked_m[G] int32; outputs with a leading G, new ones zero on the rows without
    data."""
    if a.dim() != 3 or b.dim() != 4:
        raise ValueError("a[G, M_cap, K], b[G, 2, I, K]")
    G, M = a.shape[:2]
    ld = (M + 3) // 4 * 4
    p, act_id, ret, I, K, suffix, index = _gated_args(a, sfa, b, sfb, act, h, q, sf, gu, (G,), (G,), M, ld)
    counts = _pointers(index, ("masked_m",), masked_m, _I32, (G,))
    _call("dg_m_grouped_fp8_gated_gemm_nt_masked" + suffix, p[0], p[1], p[2], p[3], act_id, p[4], p[5], p[6], p[7],
          counts[0], G, M, I, K, int(expected_m), _raw_stream(index))
    return ret


_GATED_BWD_NAMES = ("gu", "dh", "m_indices", "dgu", "q", "sf", "qt", "sft", "ht", "sfht")


def gated_backward_quantize_e4m3(gu, dh, act="silu", m_indices=None, dgu=None, q=None, sf=None, qt=None, sft=None,
                                 ht=None, sfht=None, ue8m0=False):
    """Gradient of h = act(gate) * up, quantised (dg_gated_backward_quantize_e4m3[_ue8m0]): gu[rows, 2I] and
    dh[rows, I] bf16, m_indices[rows] int32 or None (rows with a negative index count as zeros).  Outputs, each a
    tensor to fill or True for a new one (scales are allocated with their codes): dgu[rows, 2I] bf16; q[rows, 2I] with
    sf[2I/128, ld]; qt[R, 2I] with sft[R/128, 2I] and ht[R, I] with sfht[R/128, I], R = rows up to a multiple of 128.
    Returns (dgu, q, sf, qt, sft, ht, sfht), None where not asked for."""
    if dh.dim() != 2:
        raise ValueError("dh[rows, I]")
    rows, I = dh.shape
    index = _device(dh, "dh")
    full = (rows + 127) // 128
    wide, wide_full, slim_full = (rows, 2 * I), (full * 128, 2 * I), (full * 128, I)
    f32 = torch.float32
    if True in (dgu is True, q is True, qt is True, ht is True):
        dev = dh.device
        dgu = _out(dgu, wide, torch.bfloat16, dev)
        q, qt, ht = _out(q, wide, torch.uint8, dev), _out(qt, wide_full, torch.uint8, dev), _out(ht, slim_full, torch.uint8, dev)
    if q is None:
        sf = None
    elif sf is None:
        sf = torch.zeros((2 * I // 128, (rows + 3) // 4 * 4), dtype=f32, device=dh.device)
    if qt is None:
        sft = None
    elif sft is None:
        sft = torch.empty((full, 2 * I), dtype=f32, device=dh.device)
    if ht is None:
        sfht = None
    elif sfht is None:
        sfht = torch.empty((full, I), dtype=f32, device=dh.device)
    ld = sf.shape[-1] if sf is not None else 0
    p = _pointers(index, _GATED_BWD_NAMES, gu, _BF16, (rows, 2, I) if gu.dim() == 3 else wide, dh, _BF16, (rows, I),
                  m_indices, _I32, (rows,), dgu, _BF16, wide, q, _E4M3, wide, sf, _F32, (2 * I // 128, ld),
                  qt, _E4M3, wide_full, sft, _F32, (full, 2 * I), ht, _E4M3, slim_full, sfht, _F32, (full, I))
    _call("dg_gated_backward_quantize_e4m3" + ("_ue8m0" if ue8m0 else ""), p[0], p[1], _act_of(act), p[2], p[3], p[4],
          p[5], ld, p[6], p[7], p[8], p[9], rows, I, _raw_stream(index))
    return dgu, q, sf, qt, sft, ht, sfht


def get_mk_alignment_for_contiguous_layout() -> int:
    return lib().dg_get_mk_alignment_for_contiguous_layout()


def set_mk_alignment_for_contiguous_layout(alignment: int):
    _check(lib().dg_set_mk_alignment_for_contiguous_layout(int(alignment)), "dg_set_mk_alignment_for_contiguous_layout")


def get_sf_aligned_size(mn: int) -> int:
    return lib().dg_get_sf_aligned_size(int(mn))


def set_num_cus(n: int):
    _check(lib().dg_set_num_cus(int(n)), "dg_set_num_cus")


def get_num_cus() -> int:
    v = lib().dg_get_num_cus()
    if v < 0:
        raise DGError(v, "dg_get_num_cus")
    return v


def set_kernel_family(name: str):
    """Kernel family of the GEMM entry points called from this thread: auto, pipe, persist, skinny or tiled."""
    _check(lib().dg_set_kernel_family(name.encode()), "dg_set_kernel_family")


def get_kernel_family() -> str:
    return lib().dg_get_kernel_family().decode()


def last_config() -> str:
    return lib().dg_last_config().decode()
