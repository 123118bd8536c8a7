"""ctypes binding of libcf (include/cf.h): the same entry points under the same
names, plus thin conveniences that allocate outputs and workspaces with torch.

Argument marshalling only: every step of the computation runs in libcf's CUDA
kernels.  Loading fails loudly if libcf.so has not been built; there is no
fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcf.so")

CF_OK = 0
CF_ERR_INVALID_ARG = 1
CF_ERR_UNSUPPORTED = 2
CF_ERR_MISALIGNED = 3
CF_ERR_WORKSPACE_TOO_SMALL = 4
CF_ERR_NOT_RESIDENT = 5
CF_ERR_CUDA = 6
CF_ERR_DEVICE_TIMEOUT = 7
CF_ERR_DEVICE_BOUNDS = 8
CF_ERR_NO_DEVICE = 9

CF_ACT_NONE = 0
CF_ACT_GELU_TANH = 1
CF_ACT_SILU = 2
CF_ACT_RELU = 3


class cf_tuning(ctypes.Structure):
    _fields_ = [
        ("n_slice", ctypes.c_int32),
        ("cluster_size", ctypes.c_int32),
        ("peer_max", ctypes.c_int32),
        ("max_clusters", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("stitch_mapping", ctypes.c_int32),
        ("timeout_us", ctypes.c_uint32),
        ("extra_arrivals", ctypes.c_int32),
        ("cluster_m", ctypes.c_int32),
        ("disable_pdl", ctypes.c_int32),
        ("trace", ctypes.c_void_p),
    ]


CF_TRACE_TILES = 16
CF_TRACE_EVENTS = 12
CF_TRACE_SLOTS = 4 + CF_TRACE_TILES * CF_TRACE_EVENTS
TRACE_EVENT_NAMES = ["tma_first", "tma_last", "mma_acc_free", "mma_first", "mma_done", "mma_wait_ns",
                     "epi_start", "epi_stats", "epi_cta", "epi_cluster", "epi_global", "epi_stored"]
# cf_trace_event (fused GEMM) and cf_trb_event (back-to-back GEMM) slots
(CF_TR_TMA_FIRST, CF_TR_TMA_LAST, CF_TR_MMA_ACC_FREE, CF_TR_MMA_FIRST, CF_TR_MMA_DONE, CF_TR_MMA_WAIT_NS,
 CF_TR_EPI_START, CF_TR_EPI_STATS, CF_TR_EPI_CTA, CF_TR_EPI_CLUSTER, CF_TR_EPI_GLOBAL, CF_TR_EPI_STORED) = range(12)
(CF_TRB_TMA_FIRST, CF_TRB_ML1_FIRST, CF_TRB_ML1_DONE, CF_TRB_EPI1_START, CF_TRB_EPI1_LOCAL, CF_TRB_EPI1_DONE,
 CF_TRB_ML2_START, CF_TRB_ML2_DONE, CF_TRB_EPI2_START, CF_TRB_EPI2_SENT, CF_TRB_EPI2_RECV,
 CF_TRB_EPI2_STORED) = range(12)


class cf_plan(ctypes.Structure):
    _fields_ = [
        ("n_slice", ctypes.c_int32),
        ("ctas_per_row", ctypes.c_int32),
        ("cluster_size", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("leader_mode", ctypes.c_int32),
        ("row_blocks", ctypes.c_int32),
        ("clusters", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32),
        ("cluster_m", ctypes.c_int32),
        ("staging_buffers", ctypes.c_int32),
    ]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class CfError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})"
                         + (f", cudaError {cf_last_cuda_error()}" if status == CF_ERR_CUDA else ""))


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_ST = ctypes.c_int

# name -> (restype, argtypes)
_SIGS = {
    "cf_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cf_version": (ctypes.c_int, []),
    "cf_last_cuda_error": (ctypes.c_int, []),
    "cf_tuning_default": (None, [ctypes.POINTER(cf_tuning)]),
    "cf_plan_gemm_fused": (_ST, [_I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                 ctypes.POINTER(cf_tuning), ctypes.POINTER(cf_plan)]),
    "cf_query_gemm_fused_plan": (_ST, [_I64, _I64, _I64, ctypes.c_int32, ctypes.POINTER(cf_tuning),
                                       ctypes.POINTER(cf_plan), ctypes.POINTER(ctypes.c_int32)]),
    "cf_gemm_fused_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "cf_stitch_workspace_size": (_SZ, [_I64, _I64]),
    "cf_workspace_init": (_ST, [_P, _SZ, _P]),
    "cf_get_device_status": (_ST, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "cf_gemm_fused_rownorm": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                    _P, _SZ, _P]),
    "cf_gemm_fused_rownorm_ex": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                       _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_gemm_fused_rownorm_noalloc": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                            _P]),
    "cf_gemm_fused_rownorm_noalloc_status": (_ST, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "cf_gemm_fused_rmsnorm": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                    _P, _SZ, _P]),
    "cf_gemm_fused_rmsnorm_ex": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                       _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_gemm_fused_residual_norm": (_ST, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                          ctypes.c_int, _P, _SZ, _P]),
    "cf_gemm_fused_residual_norm_ex": (_ST, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                             ctypes.c_int, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_gemm_fused_rowsoftmax_causal": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _F, _I64, _P, _SZ, _P]),
    "cf_gemm_fused_rowsoftmax_causal_ex": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _F, _I64, _P, _SZ, _P,
                                                 ctypes.POINTER(cf_tuning)]),
    "cf_gemm_fused_rowsoftmax": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _F, _P, _SZ, _P]),
    "cf_gemm_fused_rowsoftmax_ex": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _F, _P, _SZ, _P,
                                          ctypes.POINTER(cf_tuning)]),
    "cf_unfused_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "cf_unfused_gemm_rownorm": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                      _P, _SZ, _P]),
    "cf_unfused_gemm_rmsnorm": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                      _P, _SZ, _P]),
    "cf_unfused_gemm_residual_norm": (_ST, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _F, _F, ctypes.c_int,
                                            ctypes.c_int, _P, _SZ, _P]),
    "cf_unfused_gemm_rowsoftmax": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _F, _P, _SZ, _P]),
    "cf_b2b_workspace_size": (_SZ, []),
    "cf_query_b2b_plan": (_ST, [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(cf_tuning),
                                ctypes.POINTER(cf_plan)]),
    "cf_b2b_gemm": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, ctypes.c_int, _P, _SZ, _P]),
    "cf_b2b_gemm_ex": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, ctypes.c_int, _P, _SZ, _P,
                             ctypes.POINTER(cf_tuning)]),
    "cf_b2b_gemm_layernorm": (_ST, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, _F, _P, _SZ, _P]),
    "cf_b2b_gemm_layernorm_ex": (_ST, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F, _F, _P, _SZ, _P,
                                       ctypes.POINTER(cf_tuning)]),
    "cf_stitch_add_layernorm": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _F, _P, _SZ, _P]),
    "cf_stitch_add_layernorm_ex": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _F, _P, _SZ, _P,
                                         ctypes.POINTER(cf_tuning)]),
    "cf_stitch_batchnorm_workspace_size": (_SZ, [_I64, _I64]),
    "cf_stitch_batchnorm": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, _SZ, _P]),
    "cf_stitch_batchnorm_ex": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, _SZ, _P,
                                     ctypes.POINTER(cf_tuning)]),
    "cf_query_stitch_batchnorm_plan": (_ST, [_I64, _I64, ctypes.POINTER(cf_tuning), ctypes.POINTER(ctypes.c_int32),
                                             ctypes.POINTER(ctypes.c_int32)]),
    "cf_stitch_rowreduce_broadcast": (_ST, [_P, _P, _P, _I64, _I64, _P, _SZ, _P]),
    "cf_stitch_rowreduce_broadcast_ex": (_ST, [_P, _P, _P, _I64, _I64, _P, _SZ, _P,
                                               ctypes.POINTER(cf_tuning)]),
    "cf_grouped_gemm_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "cf_grouped_gemm": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _SZ, _P]),
    "cf_grouped_gemm_ex": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _SZ, _P,
                                 ctypes.POINTER(cf_tuning)]),
    "cf_grouped_gemm_dgrad": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, _P, _SZ, _P]),
    "cf_grouped_gemm_dgrad_ex": (_ST, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, _P, _SZ, _P,
                                       ctypes.POINTER(cf_tuning)]),
    "cf_grouped_gemm_wgrad": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, _P, _SZ, _P]),
    "cf_grouped_gemm_wgrad_ex": (_ST, [_P, _P, _P, _P, _I64, _I64, _I64, _I64, ctypes.c_int, _P, _SZ, _P,
                                       ctypes.POINTER(cf_tuning)]),
    "cf_gemm_lora_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "cf_gemm_lora": (_ST, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.c_int, _P,
                           _SZ, _P]),
    "cf_gemm_lora_ex": (_ST, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, ctypes.c_int,
                              _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_gemm_linear_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "cf_gemm_linear": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _SZ, _P]),
    "cf_gemm_linear_ex": (_ST, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _SZ, _P,
                                ctypes.POINTER(cf_tuning)]),
    "cf_gemm_linear_grad": (_ST, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P,
                                  _SZ, _P]),
    "cf_gemm_linear_grad_ex": (_ST, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P,
                                     _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_stitch_block_norms": (_ST, [_P] * 9 + [_I64] * 3 + [ctypes.c_int] * 2 + [_F] * 3 + [ctypes.c_int, _P, _SZ, _P]),
    "cf_stitch_block_norms_ex": (_ST, [_P] * 9 + [_I64] * 3 + [ctypes.c_int] * 2 + [_F] * 3 +
                                 [ctypes.c_int, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_stitch_block_norms_grad_workspace_size": (_SZ, [_I64, _I64]),
    "cf_stitch_block_norms_grad": (_ST, [_P] * 15 + [_I64] * 3 + [ctypes.c_int] * 2 + [_F] * 3 +
                                   [ctypes.c_int, _P, _SZ, _P]),
    "cf_stitch_block_norms_grad_ex": (_ST, [_P] * 15 + [_I64] * 3 + [ctypes.c_int] * 2 + [_F] * 3 +
                                      [ctypes.c_int, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_stitch_logprobs": (_ST, [_P] * 7 + [_I64] * 4 + [_F, ctypes.c_int, _P, _SZ, _P]),
    "cf_stitch_logprobs_ex": (_ST, [_P] * 7 + [_I64] * 4 + [_F, ctypes.c_int, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_stitch_logprobs_grad": (_ST, [_P] * 8 + [_I64] * 4 + [_F, ctypes.c_int, _P, _SZ, _P]),
    "cf_stitch_logprobs_grad_ex": (_ST, [_P] * 8 + [_I64] * 4 +
                                   [_F, ctypes.c_int, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
    "cf_stitch_powadd_softmax": (_ST, [_P, _P, _F, _P, _I64, _I64, _P, _SZ, _P]),
    "cf_stitch_powadd_softmax_ex": (_ST, [_P, _P, _F, _P, _I64, _I64, _P, _SZ, _P, ctypes.POINTER(cf_tuning)]),
}

_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libcf.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"libcf.so not built at {LIB_PATH}; run "
                                  "`python -m memory_fusion_gb300.build` (no fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def declared_symbols():
    return list(_SIGS)


# ---------------------------------------------------------------------------
# raw entry points (same names and argument order as the C ABI)
# ---------------------------------------------------------------------------
def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        raise TypeError(f"cannot pass {type(x)} as a pointer") from None


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _tun(t):
    return None if t is None else ctypes.byref(t)


def status_string(status: int) -> str:
    return lib().cf_status_string(int(status)).decode()


def cf_version() -> int:
    return lib().cf_version()


def cf_last_cuda_error() -> int:
    return lib().cf_last_cuda_error()


def cf_tuning_default() -> cf_tuning:
    t = cf_tuning()
    lib().cf_tuning_default(ctypes.byref(t))
    return t


def cf_plan_gemm_fused(M, N, K, sm_count, max_active_clusters, tuning=None):
    """max_active_clusters: 17 ints, index = cluster size (entry 0 unused)."""
    if len(max_active_clusters) != 17:
        raise ValueError("max_active_clusters needs 17 entries (index = cluster size)")
    arr = (ctypes.c_int32 * 17)(*[int(v) for v in max_active_clusters])
    p = cf_plan()
    st = lib().cf_plan_gemm_fused(M, N, K, sm_count, arr, _tun(tuning), ctypes.byref(p))
    return st, p


def cf_query_gemm_fused_plan(M, N, K, kind, tuning=None):
    """(status, plan, max_active_clusters[17]) on the current device; kind 0 LN, 1 GELU+LN, 2 softmax."""
    p = cf_plan()
    arr = (ctypes.c_int32 * 17)()
    st = lib().cf_query_gemm_fused_plan(M, N, K, kind, _tun(tuning), ctypes.byref(p), arr)
    return st, p, list(arr)


def cf_gemm_fused_workspace_size(M, N, K) -> int:
    return lib().cf_gemm_fused_workspace_size(M, N, K)


def cf_stitch_workspace_size(rows, cols) -> int:
    return lib().cf_stitch_workspace_size(rows, cols)


def cf_workspace_init(ws, nbytes, stream=None) -> int:
    return lib().cf_workspace_init(_ptr(ws), nbytes, _stream(stream))


def cf_get_device_status(ws, stream=None):
    info = ctypes.c_int32(0)
    st = lib().cf_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(info))
    return st, info.value


def cf_gemm_fused_rownorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, act, workspace,
                          workspace_bytes, stream=None, tuning=None) -> int:
    L = lib()
    if tuning is None:
        return L.cf_gemm_fused_rownorm(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                       M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                       _stream(stream))
    return L.cf_gemm_fused_rownorm_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                      M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                      _stream(stream), _tun(tuning))


def cf_gemm_fused_rmsnorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, act, workspace,
                          workspace_bytes, stream=None, tuning=None) -> int:
    """Y = RMSNorm(act(alpha*X.W + bias)) * gamma (+ beta); beta may be None."""
    L = lib()
    if tuning is None:
        return L.cf_gemm_fused_rmsnorm(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                       M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                       _stream(stream))
    return L.cf_gemm_fused_rmsnorm_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                      M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                      _stream(stream), _tun(tuning))


CF_NORM_LAYER = 0
CF_NORM_RMS = 1
CF_NORM_NONE = 2


def cf_gemm_fused_residual_norm(X, W, bias, R, gamma, beta, Y, M, N, K, alpha, eps, act, norm, workspace,
                                workspace_bytes, stream=None, tuning=None) -> int:
    """Y = Norm(act(alpha*X.W + bias) + R) * gamma (+ beta); norm CF_NORM_LAYER or CF_NORM_RMS."""
    L = lib()
    if tuning is None:
        return L.cf_gemm_fused_residual_norm(_ptr(X), _ptr(W), _ptr(bias), _ptr(R), _ptr(gamma), _ptr(beta),
                                             _ptr(Y), M, N, K, alpha, eps, act, norm, _ptr(workspace),
                                             workspace_bytes, _stream(stream))
    return L.cf_gemm_fused_residual_norm_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(R), _ptr(gamma), _ptr(beta),
                                            _ptr(Y), M, N, K, alpha, eps, act, norm, _ptr(workspace),
                                            workspace_bytes, _stream(stream), _tun(tuning))


def cf_unfused_gemm_residual_norm(X, W, bias, R, gamma, beta, Y, M, N, K, alpha, eps, act, norm, workspace,
                                  workspace_bytes, stream=None) -> int:
    return lib().cf_unfused_gemm_residual_norm(_ptr(X), _ptr(W), _ptr(bias), _ptr(R), _ptr(gamma), _ptr(beta),
                                               _ptr(Y), M, N, K, alpha, eps, act, norm, _ptr(workspace),
                                               workspace_bytes, _stream(stream))


def cf_gemm_fused_rownorm_noalloc(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, act, stream=None) -> int:
    """cf_gemm_fused_rownorm without a workspace: for callers that cannot
    allocate device memory; its scratch is a fixed 4 MiB array inside libcf."""
    return lib().cf_gemm_fused_rownorm_noalloc(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                               M, N, K, alpha, eps, act, _stream(stream))


def cf_gemm_fused_rownorm_noalloc_status(stream=None):
    """(status, info) of the no-allocation calls on the current device: waits
    for the stream, reads and clears the fixed scratch array's error word."""
    info = ctypes.c_int32(0)
    st = lib().cf_gemm_fused_rownorm_noalloc_status(_stream(stream), ctypes.byref(info))
    return st, info.value


def cf_gemm_fused_rowsoftmax(X, W, bias, Y, M, N, K, scale, workspace, workspace_bytes,
                             stream=None, tuning=None) -> int:
    L = lib()
    if tuning is None:
        return L.cf_gemm_fused_rowsoftmax(_ptr(X), _ptr(W), _ptr(bias), _ptr(Y), M, N, K, scale,
                                          _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_gemm_fused_rowsoftmax_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(Y), M, N, K, scale,
                                         _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_stitch_rowreduce_broadcast(A, row_bias, out, rows, cols, workspace, workspace_bytes,
                                  stream=None, tuning=None) -> int:
    L = lib()
    if tuning is None:
        return L.cf_stitch_rowreduce_broadcast(_ptr(A), _ptr(row_bias), _ptr(out), rows, cols,
                                               _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_stitch_rowreduce_broadcast_ex(_ptr(A), _ptr(row_bias), _ptr(out), rows, cols,
                                              _ptr(workspace), workspace_bytes, _stream(stream),
                                              _tun(tuning))


def cf_stitch_powadd_softmax(A, w, p, out, rows, cols, workspace, workspace_bytes, stream=None, tuning=None) -> int:
    L = lib()
    if tuning is None:
        return L.cf_stitch_powadd_softmax(_ptr(A), _ptr(w), p, _ptr(out), rows, cols, _ptr(workspace),
                                          workspace_bytes, _stream(stream))
    return L.cf_stitch_powadd_softmax_ex(_ptr(A), _ptr(w), p, _ptr(out), rows, cols, _ptr(workspace),
                                         workspace_bytes, _stream(stream), _tun(tuning))


def cf_unfused_workspace_size(M, N, K) -> int:
    return lib().cf_unfused_workspace_size(M, N, K)


def cf_unfused_gemm_rownorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, act, workspace, workspace_bytes,
                            stream=None) -> int:
    """The unfused two-kernel composition (GEMM -> fp32 P -> row kernel), for comparison."""
    return lib().cf_unfused_gemm_rownorm(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                         M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                         _stream(stream))


def cf_gemm_fused_rowsoftmax_causal(X, W, bias, Y, M, N, K, scale, offset, workspace, workspace_bytes,
                                    stream=None, tuning=None) -> int:
    """Y = softmax over each row of scale*X.W + bias keeping column j of row i iff j <= i + offset."""
    L = lib()
    if tuning is None:
        return L.cf_gemm_fused_rowsoftmax_causal(_ptr(X), _ptr(W), _ptr(bias), _ptr(Y), M, N, K, scale, offset,
                                                 _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_gemm_fused_rowsoftmax_causal_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(Y), M, N, K, scale, offset,
                                                _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_unfused_gemm_rmsnorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, act, workspace, workspace_bytes,
                            stream=None) -> int:
    return lib().cf_unfused_gemm_rmsnorm(_ptr(X), _ptr(W), _ptr(bias), _ptr(gamma), _ptr(beta), _ptr(Y),
                                         M, N, K, alpha, eps, act, _ptr(workspace), workspace_bytes,
                                         _stream(stream))


def cf_unfused_gemm_rowsoftmax(X, W, bias, Y, M, N, K, scale, workspace, workspace_bytes, stream=None) -> int:
    return lib().cf_unfused_gemm_rowsoftmax(_ptr(X), _ptr(W), _ptr(bias), _ptr(Y), M, N, K, scale,
                                            _ptr(workspace), workspace_bytes, _stream(stream))


CF_B2B_SOFTMAX = 0
CF_B2B_GELU_TANH = 1
CF_B2B_LAYERNORM = 2


def cf_b2b_workspace_size() -> int:
    return lib().cf_b2b_workspace_size()


def cf_query_b2b_plan(M, K, N1, N2, op, tuning=None):
    """(status, plan) of the back-to-back GEMM launch on the current device."""
    p = cf_plan()
    st = lib().cf_query_b2b_plan(M, K, N1, N2, op, _tun(tuning), ctypes.byref(p))
    return st, p


def cf_b2b_gemm(X, W1, b1, W2, O, M, K, N1, N2, alpha, op, workspace, workspace_bytes, stream=None,
                tuning=None) -> int:
    """O = bf16(F(alpha*X.W1 + b1)) . W2 with F the row softmax (op 0) or GELU_tanh (op 1)."""
    L = lib()
    if tuning is None:
        return L.cf_b2b_gemm(_ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(O), M, K, N1, N2, alpha, op,
                             _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_b2b_gemm_ex(_ptr(X), _ptr(W1), _ptr(b1), _ptr(W2), _ptr(O), M, K, N1, N2, alpha, op,
                            _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def check(status: int, what: str = "libcf"):
    if status != CF_OK:
        raise CfError(status, what)


# ---------------------------------------------------------------------------
# conveniences over torch tensors (allocation in Python, compute in libcf)
# ---------------------------------------------------------------------------
def tuning(**kw) -> cf_tuning:
    t = cf_tuning_default()
    for k, v in kw.items():
        setattr(t, k, v.data_ptr() if k == "trace" and hasattr(v, "data_ptr") else v)
    return t


def new_workspace(nbytes: int, device=None, stream=None):
    import torch
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")
    check(cf_workspace_init(ws, ws.numel(), stream), "cf_workspace_init")
    return ws


def gemm_fused_rownorm(X, W, bias, gamma, beta, *, alpha=1.0, eps=1e-5, act="none", out=None,
                       workspace=None, stream=None, tuning=None):
    """Y = LayerNorm(act(alpha*X@W + bias))*gamma + beta; X, W bf16 CUDA tensors."""
    import torch
    M, K = X.shape
    N = W.shape[1]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_gemm_fused_workspace_size(M, N, K),
                                                               X.device, stream)
    a = {"none": CF_ACT_NONE, "gelu_tanh": CF_ACT_GELU_TANH}[act]
    check(cf_gemm_fused_rownorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, a, ws, ws.numel(),
                                stream, tuning), "cf_gemm_fused_rownorm")
    return Y


def gemm_fused_rmsnorm(X, W, bias, gamma, beta=None, *, alpha=1.0, eps=1e-5, act="none", out=None,
                       workspace=None, stream=None, tuning=None):
    """Y = RMSNorm(act(alpha*X@W + bias))*gamma (+ beta); X, W bf16 CUDA tensors."""
    import torch
    M, K = X.shape
    N = W.shape[1]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_gemm_fused_workspace_size(M, N, K),
                                                               X.device, stream)
    a = {"none": CF_ACT_NONE, "gelu_tanh": CF_ACT_GELU_TANH}[act]
    check(cf_gemm_fused_rmsnorm(X, W, bias, gamma, beta, Y, M, N, K, alpha, eps, a, ws, ws.numel(),
                                stream, tuning), "cf_gemm_fused_rmsnorm")
    return Y


def gemm_fused_rowsoftmax(X, W, bias=None, *, scale=1.0, out=None, workspace=None, stream=None,
                          tuning=None):
    """Y = softmax(scale*X@W + bias) over rows; X, W bf16 CUDA tensors."""
    import torch
    M, K = X.shape
    N = W.shape[1]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_gemm_fused_workspace_size(M, N, K),
                                                               X.device, stream)
    check(cf_gemm_fused_rowsoftmax(X, W, bias, Y, M, N, K, scale, ws, ws.numel(), stream, tuning),
          "cf_gemm_fused_rowsoftmax")
    return Y


def gemm_fused_residual_norm(X, W, bias, R, gamma, beta=None, *, alpha=1.0, eps=1e-5, act="none", norm="layer",
                             out=None, workspace=None, stream=None, tuning=None):
    """Y = Norm(act(alpha*X@W + bias) + R)*gamma (+ beta), Norm = "layer" or "rms"; X, W, R bf16 CUDA tensors."""
    import torch
    M, K = X.shape
    N = W.shape[1]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_gemm_fused_workspace_size(M, N, K),
                                                               X.device, stream)
    a = {"none": CF_ACT_NONE, "gelu_tanh": CF_ACT_GELU_TANH}[act]
    n = {"layer": CF_NORM_LAYER, "rms": CF_NORM_RMS}[norm]
    check(cf_gemm_fused_residual_norm(X, W, bias, R, gamma, beta, Y, M, N, K, alpha, eps, a, n, ws, ws.numel(),
                                      stream, tuning), "cf_gemm_fused_residual_norm")
    return Y


def gemm_fused_rowsoftmax_causal(X, W, bias=None, *, scale=1.0, offset=0, out=None, workspace=None, stream=None,
                                 tuning=None):
    """Y = softmax over each row of scale*X@W + bias keeping column j of row i iff j <= i + offset."""
    import torch
    M, K = X.shape
    N = W.shape[1]
    Y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_gemm_fused_workspace_size(M, N, K),
                                                               X.device, stream)
    check(cf_gemm_fused_rowsoftmax_causal(X, W, bias, Y, M, N, K, scale, offset, ws, ws.numel(), stream, tuning),
          "cf_gemm_fused_rowsoftmax_causal")
    return Y


def cf_b2b_gemm_layernorm(X, W1, b1, gamma1, beta1, W2, O, M, K, N1, N2, alpha, eps, workspace, workspace_bytes,
                          stream=None, tuning=None) -> int:
    """O = bf16(LayerNorm(alpha*X.W1 + b1)*gamma1 + beta1) . W2 (LayerNorm over the N1 columns)."""
    L = lib()
    if tuning is None:
        return L.cf_b2b_gemm_layernorm(_ptr(X), _ptr(W1), _ptr(b1), _ptr(gamma1), _ptr(beta1), _ptr(W2), _ptr(O),
                                       M, K, N1, N2, alpha, eps, _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_b2b_gemm_layernorm_ex(_ptr(X), _ptr(W1), _ptr(b1), _ptr(gamma1), _ptr(beta1), _ptr(W2), _ptr(O),
                                      M, K, N1, N2, alpha, eps, _ptr(workspace), workspace_bytes, _stream(stream),
                                      _tun(tuning))


def cf_stitch_add_layernorm(A, R, gamma, beta, out, rows, cols, eps, workspace, workspace_bytes, stream=None,
                            tuning=None) -> int:
    """out = LayerNorm(A + R) * gamma + beta over each row (R may be None)."""
    L = lib()
    if tuning is None:
        return L.cf_stitch_add_layernorm(_ptr(A), _ptr(R), _ptr(gamma), _ptr(beta), _ptr(out), rows, cols, eps,
                                         _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_stitch_add_layernorm_ex(_ptr(A), _ptr(R), _ptr(gamma), _ptr(beta), _ptr(out), rows, cols, eps,
                                        _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_stitch_batchnorm_workspace_size(rows, cols) -> int:
    return lib().cf_stitch_batchnorm_workspace_size(rows, cols)


def cf_stitch_batchnorm(A, gamma, beta, out, mean_out, var_out, rows, cols, eps, workspace, workspace_bytes,
                        stream=None, tuning=None) -> int:
    """out = (A - mean_col)/sqrt(var_col + eps)*gamma + beta with batch statistics over the rows."""
    L = lib()
    if tuning is None:
        return L.cf_stitch_batchnorm(_ptr(A), _ptr(gamma), _ptr(beta), _ptr(out), _ptr(mean_out), _ptr(var_out),
                                     rows, cols, eps, _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_stitch_batchnorm_ex(_ptr(A), _ptr(gamma), _ptr(beta), _ptr(out), _ptr(mean_out), _ptr(var_out),
                                    rows, cols, eps, _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_query_stitch_batchnorm_plan(rows, cols, tuning=None):
    """(status, mapping 3 Regional / 4 Global, grid) on the current device."""
    m, g = ctypes.c_int32(0), ctypes.c_int32(0)
    st = lib().cf_query_stitch_batchnorm_plan(rows, cols, _tun(tuning), ctypes.byref(m), ctypes.byref(g))
    return st, m.value, g.value


def stitch_add_layernorm(A, R, gamma, beta, *, eps=1e-5, out=None, workspace=None, stream=None, tuning=None):
    """LayerNorm(A + R) * gamma + beta over rows; fp32 CUDA tensors (R may be None)."""
    import torch
    rows, cols = A.shape
    O = out if out is not None else torch.empty_like(A)
    ws = workspace if workspace is not None else new_workspace(cf_stitch_workspace_size(rows, cols), A.device,
                                                               stream)
    check(cf_stitch_add_layernorm(A, R, gamma, beta, O, rows, cols, eps, ws, ws.numel(), stream, tuning),
          "cf_stitch_add_layernorm")
    return O


def stitch_batchnorm(A, gamma, beta, *, eps=1e-5, out=None, workspace=None, stream=None, tuning=None):
    """(out, mean, var): BatchNorm of fp32 A [rows, cols] with its batch statistics."""
    import torch
    rows, cols = A.shape
    O = out if out is not None else torch.empty_like(A)
    mean = torch.empty(cols, dtype=torch.float32, device=A.device)
    var = torch.empty(cols, dtype=torch.float32, device=A.device)
    ws = workspace if workspace is not None else new_workspace(cf_stitch_batchnorm_workspace_size(rows, cols),
                                                               A.device, stream)
    check(cf_stitch_batchnorm(A, gamma, beta, O, mean, var, rows, cols, eps, ws, ws.numel(), stream, tuning),
          "cf_stitch_batchnorm")
    return O, mean, var


def b2b_gemm(X, W1, W2, b1=None, *, op="softmax", alpha=1.0, gamma1=None, beta1=None, eps=1e-5, out=None,
             workspace=None, stream=None, tuning=None):
    """O = bf16(F(alpha*X@W1 + b1)) @ W2, F = "softmax" (rows), "gelu_tanh" or "layernorm" (rows, with
    gamma1, beta1); bf16 CUDA tensors."""
    import torch
    ops = {"softmax": CF_B2B_SOFTMAX, "gelu_tanh": CF_B2B_GELU_TANH, "layernorm": CF_B2B_LAYERNORM}
    if op not in ops:
        raise ValueError(f"unknown op {op!r}")
    M, K = X.shape
    N1 = W1.shape[1]
    N2 = W2.shape[1]
    O = out if out is not None else torch.empty((M, N2), dtype=torch.bfloat16, device=X.device)
    ws = workspace if workspace is not None else new_workspace(cf_b2b_workspace_size(), X.device, stream)
    if op == "layernorm":
        check(cf_b2b_gemm_layernorm(X, W1, b1, gamma1, beta1, W2, O, M, K, N1, N2, alpha, eps, ws, ws.numel(),
                                    stream, tuning), "cf_b2b_gemm_layernorm")
    else:
        check(cf_b2b_gemm(X, W1, b1, W2, O, M, K, N1, N2, alpha, ops[op], ws, ws.numel(), stream, tuning),
              "cf_b2b_gemm")
    return O


def stitch_rowreduce_broadcast(A, row_bias, *, out=None, workspace=None, stream=None, tuning=None):
    """out = softmax_row(A^3 + row_bias[:, None]); fp32 CUDA tensors."""
    import torch
    rows, cols = A.shape
    O = out if out is not None else torch.empty_like(A)
    ws = workspace if workspace is not None else new_workspace(cf_stitch_workspace_size(rows, cols),
                                                               A.device, stream)
    check(cf_stitch_rowreduce_broadcast(A, row_bias, O, rows, cols, ws, ws.numel(), stream, tuning),
          "cf_stitch_rowreduce_broadcast")
    return O


def stitch_powadd_softmax(A, w, p, *, out=None, workspace=None, stream=None, tuning=None):
    """out = softmax_row(A + w[None, :] ** p) (w > 0); fp32 CUDA tensors."""
    import torch
    rows, cols = A.shape
    O = out if out is not None else torch.empty_like(A)
    ws = workspace if workspace is not None else new_workspace(cf_stitch_workspace_size(rows, cols),
                                                               A.device, stream)
    check(cf_stitch_powadd_softmax(A, w, float(p), O, rows, cols, ws, ws.numel(), stream, tuning),
          "cf_stitch_powadd_softmax")
    return O


# ---------------------------------------------------------------------------
# grouped GEMM and low-rank adapters
# ---------------------------------------------------------------------------
CF_BF16 = 0
CF_FP16 = 1
CF_FP32 = 2


def cf_grouped_gemm_workspace_size(T, N, K, E) -> int:
    return lib().cf_grouped_gemm_workspace_size(T, N, K, E)


def cf_grouped_gemm(X, W, offsets, Y, Z, T, N, K, E, dtype, act, workspace, workspace_bytes, stream=None,
                    tuning=None) -> int:
    """Y = act(X . W[e]) for the rows of each group e; Z (or None) receives the pre-activation."""
    L = lib()
    if tuning is None:
        return L.cf_grouped_gemm(_ptr(X), _ptr(W), _ptr(offsets), _ptr(Y), _ptr(Z), T, N, K, E, dtype, act,
                                 _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_grouped_gemm_ex(_ptr(X), _ptr(W), _ptr(offsets), _ptr(Y), _ptr(Z), T, N, K, E, dtype, act,
                                _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_grouped_gemm_dgrad(dY, W, offsets, Z, dX, T, N, K, E, dtype, workspace, workspace_bytes, stream=None,
                          tuning=None) -> int:
    """dX = (dY . W[e]^T) * act'(Z) for the rows of each group e (Z may be None)."""
    L = lib()
    if tuning is None:
        return L.cf_grouped_gemm_dgrad(_ptr(dY), _ptr(W), _ptr(offsets), _ptr(Z), _ptr(dX), T, N, K, E, dtype,
                                       _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_grouped_gemm_dgrad_ex(_ptr(dY), _ptr(W), _ptr(offsets), _ptr(Z), _ptr(dX), T, N, K, E, dtype,
                                      _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_grouped_gemm_wgrad(X, dY, offsets, dW, T, N, K, E, dtype, workspace, workspace_bytes, stream=None,
                          tuning=None) -> int:
    """dW[e] = X^T . dY over the rows of each group e."""
    L = lib()
    if tuning is None:
        return L.cf_grouped_gemm_wgrad(_ptr(X), _ptr(dY), _ptr(offsets), _ptr(dW), T, N, K, E, dtype,
                                       _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_grouped_gemm_wgrad_ex(_ptr(X), _ptr(dY), _ptr(offsets), _ptr(dW), T, N, K, E, dtype,
                                      _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_gemm_lora_workspace_size(T, N, K, S, R) -> int:
    return lib().cf_gemm_lora_workspace_size(T, N, K, S, R)


def cf_gemm_lora(X, W, bias, A, B, offsets, adapters, scale, Y, T, N, K, S, L, R, dtype, workspace, workspace_bytes,
                 stream=None, tuning=None) -> int:
    """Y = X . W + bias + scale[a] * (X . A[a]) . B[a], a the adapter of the row's request (-1: none)."""
    lb = lib()
    if tuning is None:
        return lb.cf_gemm_lora(_ptr(X), _ptr(W), _ptr(bias), _ptr(A), _ptr(B), _ptr(offsets), _ptr(adapters),
                               _ptr(scale), _ptr(Y), T, N, K, S, L, R, dtype, _ptr(workspace), workspace_bytes,
                               _stream(stream))
    return lb.cf_gemm_lora_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(A), _ptr(B), _ptr(offsets), _ptr(adapters),
                              _ptr(scale), _ptr(Y), T, N, K, S, L, R, dtype, _ptr(workspace), workspace_bytes,
                              _stream(stream), _tun(tuning))


_ACTS = {"none": CF_ACT_NONE, "gelu_tanh": CF_ACT_GELU_TANH}
_DTYPES = {}  # torch.bfloat16 and float16, once torch is there


def _first(name, t, dims):
    """Sizes, device and dtype of the tensor that the others have to agree with, and the library's name of its dtype."""
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        import torch
        _DTYPES.update({torch.bfloat16: CF_BF16, torch.float16: CF_FP16})
        dt = _DTYPES.get(t.dtype)
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, not on a CUDA device")
    if dt is None:
        raise ValueError(f"{name} has dtype {t.dtype}, not bfloat16 or float16")
    shape = _sizes(name, t, dims)
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")
    return shape, t.device, t.dtype, dt


def _sizes(name, t, dims):
    """The sizes of a tensor that has to have `dims` of them."""
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} has {len(shape)} dimensions, not {dims}")
    return shape


def _operand(name, t, shape, dtype, device):
    """The address of a tensor argument (None: none), checked against its whole shape."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{name} is not contiguous")


def _int32():
    import torch
    return torch.int32


@contextlib.contextmanager
def _launch_on(device, stream):
    """The operands' device, and `stream` (a torch stream or a handle; None = the device's current one), made current:
    outputs and workspaces allocated inside belong to the stream that uses them."""
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            if not isinstance(stream, int):
                s = stream
            elif stream in (0, 1):  # the legacy default stream (torch makes a stream of its own for an external 0)
                s = torch.cuda.default_stream(device)
            else:
                s = torch.cuda.ExternalStream(stream, device=device)
            with torch.cuda.stream(s):
                yield


def _run(name, before, between, out, shape, dtype, device, workspace, size, sizes, stream, tuning):
    """name(*before, out, *between, workspace, its bytes, stream) on the operands' device, with the output and the
    workspace (size(*sizes) bytes) made where none are given; the output.  (Written for the decode step, whose kernel
    takes less time than the host does for its call.)"""
    import torch
    index = device.index
    if workspace is not None and not (workspace.get_device() == index and workspace.is_contiguous()):
        raise ValueError(f"workspace is not a contiguous tensor on {device}")
    if stream is not None and getattr(stream, "device", device) != device:
        raise ValueError(f"stream is on {stream.device}, not on {device}")
    if stream is not None or index != torch._C._cuda_getDevice():
        with _launch_on(device, stream):
            return _run(name, before, between, out, shape, dtype, device, workspace, size, sizes, None, tuning)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        at = out.data_ptr()
    else:
        at = _operand("out", out, shape, dtype, device)
    if workspace is None:
        workspace = new_workspace(size(*sizes), device)
    last = (workspace.data_ptr(), workspace.nbytes, torch._C._cuda_getCurrentRawStream(index))
    if tuning is None:
        st = getattr(lib(), name)(*before, at, *between, *last)
    else:
        st = getattr(lib(), name + "_ex")(*before, at, *between, *last, ctypes.byref(tuning))
    if st != CF_OK:
        raise CfError(st, name)
    return out


def _act(act):
    a = _ACTS.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}")
    return a


def grouped_gemm(X, W, offsets, *, act="none", preact=None, out=None, workspace=None, stream=None, tuning=None):
    """Y[r] = act(X[r] @ W[e]) for the rows r in [offsets[e], offsets[e+1]); X [T, K] and W [E, K, N] bf16 or fp16
    CUDA tensors, offsets int32 [E + 1] on the same device.  `preact` ([T, N]) receives the unactivated product for
    grouped_gemm_dgrad.  Rows of no group are not written: in a new output they hold anything."""
    (T, K), dev, dtype, dt = _first("X", X, 2)
    a = _act(act)
    E, _, N = _sizes("W", W, 3)
    before = (X.data_ptr(), _operand("W", W, (E, K, N), dtype, dev),
              _operand("offsets", offsets, (E + 1,), _int32(), dev))
    between = (_operand("preact", preact, (T, N), dtype, dev), T, N, K, E, dt, a)
    return _run("cf_grouped_gemm", before, between, out, (T, N), dtype, dev, workspace,
                cf_grouped_gemm_workspace_size, (T, N, K, E), stream, tuning)


def grouped_gemm_dgrad(dY, W, offsets, *, preact=None, out=None, workspace=None, stream=None, tuning=None):
    """dX[r] = (dY[r] @ W[e].T) * gelu_tanh'(preact[r]) for the rows of each group; dY [T, N], W [E, K, N],
    preact [T, K] or None (no activation before these rows).  out may be preact."""
    (T, N), dev, dtype, dt = _first("dY", dY, 2)
    E, K, _ = _sizes("W", W, 3)
    before = (dY.data_ptr(), _operand("W", W, (E, K, N), dtype, dev),
              _operand("offsets", offsets, (E + 1,), _int32(), dev),
              _operand("preact", preact, (T, K), dtype, dev))
    return _run("cf_grouped_gemm_dgrad", before, (T, N, K, E, dt), out, (T, K), dtype, dev, workspace,
                cf_grouped_gemm_workspace_size, (T, N, K, E), stream, tuning)


def grouped_gemm_wgrad(X, dY, offsets, *, out=None, workspace=None, stream=None, tuning=None):
    """dW[e] = X[rows of e].T @ dY[rows of e] (zeros for an empty group), [E, K, N]; X [T, K], dY [T, N]."""
    (T, K), dev, dtype, dt = _first("X", X, 2)
    N = _sizes("dY", dY, 2)[1]
    E = _sizes("offsets", offsets, 1)[0] - 1
    if E < 0:
        raise ValueError("offsets is empty: it has one entry more than there are groups")
    before = (X.data_ptr(), _operand("dY", dY, (T, N), dtype, dev),
              _operand("offsets", offsets, (E + 1,), _int32(), dev))
    return _run("cf_grouped_gemm_wgrad", before, (T, N, K, E, dt), out, (E, K, N), dtype, dev, workspace,
                cf_grouped_gemm_workspace_size, (T, N, K, E), stream, tuning)


def gemm_lora(X, W, bias, A, B, offsets, adapters, *, scale=None, out=None, workspace=None, stream=None, tuning=None):
    """Y[r] = X[r] @ W + bias + scale[a] * (X[r] @ A[a]) @ B[a] for the rows r of request s,
    [offsets[s], offsets[s+1]), with a = adapters[s] (-1: no adapter).  X [T, K], W [K, N], A [L, K, R], B [L, R, N]
    bf16 or fp16; bias fp32 [N] or None; offsets int32 [S + 1], adapters int32 [S], scale fp32 [L] or None (1).
    fp16: values of scale[a] * X[r] @ A[a] beyond +-131,008 count as that, and the workspace's status says so."""
    import torch
    (T, K), dev, dtype, dt = _first("X", X, 2)
    N = _sizes("W", W, 2)[1]
    L, _, R = _sizes("A", A, 3)
    S = _sizes("adapters", adapters, 1)[0]
    before = (X.data_ptr(), _operand("W", W, (K, N), dtype, dev), _operand("bias", bias, (N,), torch.float32, dev),
              _operand("A", A, (L, K, R), dtype, dev), _operand("B", B, (L, R, N), dtype, dev),
              _operand("offsets", offsets, (S + 1,), torch.int32, dev),
              _operand("adapters", adapters, (S,), torch.int32, dev),
              _operand("scale", scale, (L,), torch.float32, dev))
    return _run("cf_gemm_lora", before, (T, N, K, S, L, R, dt), out, (T, N), dtype, dev, workspace,
                cf_gemm_lora_workspace_size, (T, N, K, S, R), stream, tuning)


# ---------------------------------------------------------------------------
# dense layer
# ---------------------------------------------------------------------------
def cf_gemm_linear_workspace_size(M, N, K) -> int:
    return lib().cf_gemm_linear_workspace_size(M, N, K)


def cf_gemm_linear(X, W, bias, R, Y, Z, M, N, K, dtype, act, workspace, workspace_bytes, stream=None,
                   tuning=None) -> int:
    """Y = act(X . W + bias) + R; Z (or None) receives X . W + bias."""
    L = lib()
    if tuning is None:
        return L.cf_gemm_linear(_ptr(X), _ptr(W), _ptr(bias), _ptr(R), _ptr(Y), _ptr(Z), M, N, K, dtype, act,
                                _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_gemm_linear_ex(_ptr(X), _ptr(W), _ptr(bias), _ptr(R), _ptr(Y), _ptr(Z), M, N, K, dtype, act,
                               _ptr(workspace), workspace_bytes, _stream(stream), _tun(tuning))


def cf_gemm_linear_grad(dY, X, W, Z, dZ, dX, dW, dbias, M, N, K, dtype, act, workspace, workspace_bytes, stream=None,
                        tuning=None) -> int:
    """dZ = dY * act'(Z), dX = dZ . W^T, dW = X^T . dZ, dbias = column sums of dZ (each of the last three or None)."""
    L = lib()
    if tuning is None:
        return L.cf_gemm_linear_grad(_ptr(dY), _ptr(X), _ptr(W), _ptr(Z), _ptr(dZ), _ptr(dX), _ptr(dW), _ptr(dbias),
                                     M, N, K, dtype, act, _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_gemm_linear_grad_ex(_ptr(dY), _ptr(X), _ptr(W), _ptr(Z), _ptr(dZ), _ptr(dX), _ptr(dW), _ptr(dbias),
                                    M, N, K, dtype, act, _ptr(workspace), workspace_bytes, _stream(stream),
                                    _tun(tuning))


_LINEAR_ACTS = {"none": CF_ACT_NONE, "gelu_tanh": CF_ACT_GELU_TANH, "silu": CF_ACT_SILU, "relu": CF_ACT_RELU}


# (The calls below are written for the decode step, whose kernels take less time than the host does for a call: torch and
# the library's functions are looked up once, and what a call needs on another stream or device it does in a call of its
# own.)
_torch = None
_entries = {}


def _the_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _away(device, stream):
    """Whether the call is for another stream or device than the current ones."""
    if stream is None:
        return device.index != _torch._C._cuda_getDevice()
    if getattr(stream, "device", device) != device:
        raise ValueError(f"stream is on {stream.device}, not on {device}")
    return True


def _launch(name, args, device, workspace, size, sizes, tuning):
    """name(*args, workspace, its bytes, the current stream), the workspace (size(*sizes) bytes) made if there is none."""
    index = device.index
    if workspace is None:
        workspace = new_workspace(size(*sizes), device)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace is not a contiguous tensor on {device}")
    if tuning is None:
        f = _entries.get(name)
        if f is None:
            f = _entries[name] = getattr(lib(), name)
        st = f(*args, workspace.data_ptr(), workspace.nbytes, _torch._C._cuda_getCurrentRawStream(index))
    else:
        st = getattr(lib(), name + "_ex")(*args, workspace.data_ptr(), workspace.nbytes,
                                          _torch._C._cuda_getCurrentRawStream(index), ctypes.byref(tuning))
    if st != CF_OK:
        raise CfError(st, name)


def _made(name, t, shape, dtype, device):
    """An output: the given one, checked, or a new one."""
    if t is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    _operand(name, t, shape, dtype, device)
    return t


def _made_like(name, t, like):
    """An output of an operand's shape and type, which takes less time to make."""
    if t is None:
        return _torch.empty_like(like)
    _operand(name, t, like.shape, like.dtype, like.device)
    return t


def _at(t):
    return None if t is None else t.data_ptr()


def gemm_linear(X, W, bias=None, *, act="none", residual=None, preact=None, out=None, workspace=None, stream=None,
                tuning=None):
    """Y = act(X @ W + bias) + residual; X [M, K], W [K, N] and residual [M, N] bf16 or fp16 CUDA tensors, bias fp32
    [N]; act "none", "gelu_tanh", "silu" or "relu".  `preact` ([M, N]) receives X @ W + bias for gemm_linear_grad.
    out may be residual."""
    f32 = (_torch or _the_torch()).float32
    (M, K), dev, dtype, dt = _first("X", X, 2)
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return gemm_linear(X, W, bias, act=act, residual=residual, preact=preact, out=out, workspace=workspace,
                               tuning=tuning)
    a = _LINEAR_ACTS.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}")
    N = _sizes("W", W, 2)[1]
    like = (M, N)
    w, b = _operand("W", W, (K, N), dtype, dev), _operand("bias", bias, (N,), f32, dev)
    r, z = _operand("residual", residual, like, dtype, dev), _operand("preact", preact, like, dtype, dev)
    y = _made("out", out, like, dtype, dev)
    _launch("cf_gemm_linear", (X.data_ptr(), w, b, r, y.data_ptr(), z, M, N, K, dt, a), dev, workspace,
            cf_gemm_linear_workspace_size, (M, N, K), tuning)
    return y


def gemm_linear_grad(dY, X, W, *, act="none", preact=None, input=True, weight=True, bias=True, dz=None, out=None,
                     workspace=None, stream=None, tuning=None):
    """(dX, dW, dbias) of Y = act(X @ W + bias) + residual for the gradient dY [M, N] of Y (the residual's own is dY);
    input, weight and bias say which are wanted (None in the place of the others; X may be None without weight, W
    without input).  `preact` is what gemm_linear kept, needed with an activation; `dz` ([M, N], made where not given)
    then receives dY * act'(preact), which the two products take rounded to dY's dtype, and may be preact or dY.  dbias is
    fp32, of the unrounded values.  `out`: three outputs, None for new ones."""
    f32 = (_torch or _the_torch()).float32
    (M, N), dev, dtype, dt = _first("dY", dY, 2)
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return gemm_linear_grad(dY, X, W, act=act, preact=preact, input=input, weight=weight, bias=bias, dz=dz,
                                    out=out, workspace=workspace, tuning=tuning)
    a = _LINEAR_ACTS.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}")
    if X is None and W is None:
        raise ValueError("neither X nor W is given")
    K = _sizes("X", X, 2)[1] if X is not None else _sizes("W", W, 2)[0]
    if (weight and X is None) or (input and W is None):
        raise ValueError("the weight's gradient needs X, the input's needs W")
    if (a != CF_ACT_NONE) != (preact is not None) or (a == CF_ACT_NONE and dz is not None):
        raise ValueError("preact goes with an activation, and so does dz")
    x, w = _operand("X", X, (M, K), dtype, dev), _operand("W", W, (K, N), dtype, dev)
    z = _operand("preact", preact, (M, N), dtype, dev)
    given = (None, None, None) if out is None else out
    dx = dw = db = d = None
    if input:
        dx = _made("out[0]", given[0], (M, K), dtype, dev) if X is None else _made_like("out[0]", given[0], X)
    if weight:
        dw = _made("out[1]", given[1], (K, N), dtype, dev) if W is None else _made_like("out[1]", given[1], W)
    if bias:
        db = _made("out[2]", given[2], (N,), f32, dev)
    if a != CF_ACT_NONE:
        d = _made_like("dz", dz, dY)
    _launch("cf_gemm_linear_grad", (dY.data_ptr(), x, w, z, _at(d), _at(dx), _at(dw), _at(db), M, N, K, dt, a), dev,
            workspace, cf_gemm_linear_workspace_size, (M, N, K), tuning)
    return dx, dw, db


# ---------------------------------------------------------------------------
# norms before and after a block
# ---------------------------------------------------------------------------
def cf_stitch_block_norms(h, x, gate, post_weight, post_bias, pre_weight, pre_bias, x_out, y, rows, cols, gates, post,
                          pre, scale, alpha, eps, dtype, workspace, workspace_bytes, stream=None, tuning=None) -> int:
    """x_out = alpha x + scale gate Post(h), y = Pre(x_out)."""
    L = lib()
    args = (_ptr(h), _ptr(x), _ptr(gate), _ptr(post_weight), _ptr(post_bias), _ptr(pre_weight), _ptr(pre_bias),
            _ptr(x_out), _ptr(y), rows, cols, gates, post, pre, scale, alpha, eps, dtype, _ptr(workspace),
            workspace_bytes, _stream(stream))
    return L.cf_stitch_block_norms(*args) if tuning is None else L.cf_stitch_block_norms_ex(*args, _tun(tuning))


def cf_stitch_block_norms_grad_workspace_size(rows, cols) -> int:
    return lib().cf_stitch_block_norms_grad_workspace_size(rows, cols)


def cf_stitch_block_norms_grad(dy, dx_out, h, x_out, gate, post_weight, post_bias, pre_weight, dh, dx, dgate,
                               dpost_weight, dpost_bias, dpre_weight, dpre_bias, rows, cols, gates, post, pre, scale,
                               alpha, eps, dtype, workspace, workspace_bytes, stream=None, tuning=None) -> int:
    L = lib()
    args = (_ptr(dy), _ptr(dx_out), _ptr(h), _ptr(x_out), _ptr(gate), _ptr(post_weight), _ptr(post_bias),
            _ptr(pre_weight), _ptr(dh), _ptr(dx), _ptr(dgate), _ptr(dpost_weight), _ptr(dpost_bias),
            _ptr(dpre_weight), _ptr(dpre_bias), rows, cols, gates, post, pre, scale, alpha, eps, dtype,
            _ptr(workspace), workspace_bytes, _stream(stream))
    if tuning is None:
        return L.cf_stitch_block_norms_grad(*args)
    return L.cf_stitch_block_norms_grad_ex(*args, _tun(tuning))


_NORMS = {"none": CF_NORM_NONE, "rms": CF_NORM_RMS, "layer": CF_NORM_LAYER}
_ROW_DTYPES = {}  # the 16-bit types and torch.float32, once torch is there


def _row_dtype(name, t):
    """The library's name of a row operand's dtype."""
    dt = _ROW_DTYPES.get(t.dtype)
    if dt is not None and t.is_cuda:
        return dt
    if not _ROW_DTYPES:
        torch = _torch or _the_torch()
        _ROW_DTYPES.update({torch.bfloat16: CF_BF16, torch.float16: CF_FP16, torch.float32: CF_FP32})
        return _row_dtype(name, t)
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, not on a CUDA device")
    raise ValueError(f"{name} has dtype {t.dtype}, not bfloat16, float16 or float32")


def _norm(name, kind, weight, bias):
    n = _NORMS.get(kind)
    if n is None:
        raise ValueError(f"{name}: unknown norm {kind!r}")
    if n == CF_NORM_NONE and not (weight is None and bias is None):
        raise ValueError(f"{name} is no norm, but has a weight or a bias")
    return n


def _gates(gate, rows):
    if gate is None:
        return 0
    gates = _sizes("gate", gate, 2)[0]
    if gates == 0 and rows > 0 or gates > 0 and rows % gates:
        raise ValueError(f"{gates} gates do not divide {rows} rows")
    return gates


def stitch_block_norms(h, x=None, *, post="none", post_weight=None, post_bias=None, gate=None, scale=1.0, alpha=1.0,
                       pre="none", pre_weight=None, pre_bias=None, eps=1e-5, out=None, norm_out=None, workspace=None,
                       stream=None, tuning=None):
    """(x', y): x' = alpha*x + scale*gate*Post(h), y = Pre(x') (None with pre "none"); h and x [T, N] bf16, fp16 or fp32
    CUDA tensors (x may be None: 0), gate [G, N] of that type, G a divisor of T (row r takes gate r // (T // G)), or
    None; Post and Pre "rms", "layer" or "none", weights and biases fp32 [N] or None.  `out` and `norm_out` take x'
    and y; each may be h or x."""
    torch = _torch or _the_torch()
    dt, dev, dtype, f32 = _row_dtype("h", h), h.device, h.dtype, torch.float32
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return stitch_block_norms(h, x, post=post, post_weight=post_weight, post_bias=post_bias, gate=gate,
                                      scale=scale, alpha=alpha, pre=pre, pre_weight=pre_weight, pre_bias=pre_bias,
                                      eps=eps, out=out, norm_out=norm_out, workspace=workspace, tuning=tuning)
    like = h.shape
    rows, cols = _sizes("h", h, 2)
    po, pr = _norm("post", post, post_weight, post_bias), _norm("pre", pre, pre_weight, pre_bias)
    gates, vector = _gates(gate, rows), (cols,)
    ph, px = _operand("h", h, like, dtype, dev), _operand("x", x, like, dtype, dev)
    pg = None if gate is None else _operand("gate", gate, (gates, cols), dtype, dev)
    pw = None if post_weight is None else _operand("post_weight", post_weight, vector, f32, dev)
    pb = None if post_bias is None else _operand("post_bias", post_bias, vector, f32, dev)
    qw = None if pre_weight is None else _operand("pre_weight", pre_weight, vector, f32, dev)
    qb = None if pre_bias is None else _operand("pre_bias", pre_bias, vector, f32, dev)
    y = None
    if pr != CF_NORM_NONE:
        y = torch.empty_like(h) if norm_out is None else _made("norm_out", norm_out, like, dtype, dev)
    elif norm_out is not None:
        raise ValueError("norm_out is given, but there is no norm before the next block")
    xo = torch.empty_like(h) if out is None else _made("out", out, like, dtype, dev)
    _launch("cf_stitch_block_norms", (ph, px, pg, pw, pb, qw, qb, xo.data_ptr(), None if y is None else y.data_ptr(), rows,
                                      cols, gates, po, pr, scale, alpha, eps, dt), dev, workspace,
            cf_stitch_workspace_size, (rows, cols), tuning)
    return xo, y


def stitch_block_norms_grad(dy, dx_out, h, x_out, *, post="none", post_weight=None, post_bias=None, gate=None,
                            scale=1.0, alpha=1.0, pre="none", pre_weight=None, pre_bias=None, eps=1e-5, dx=True,
                            out=None, workspace=None, stream=None, tuning=None):
    """(dh, dx, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias) of stitch_block_norms for the gradients dy of y
    and dx_out of x' ([T, N]): those of what is given there, fp32 for weights and biases, None in the place of the others
    and, with dx=False, of dx.  dy goes with a Pre norm, dx_out may then be None (0); where only x' was used, the call is
    one with pre "none" (dy None, x_out not read, no gradients of Pre's weight and bias).  h and x_out ([T, N]) are the
    forward pass's input and output.  `out`: seven outputs, None for new ones; dh and dx may be dy, dx_out, h or x_out."""
    torch = _torch or _the_torch()
    dt, dev, dtype, f32 = _row_dtype("h", h), h.device, h.dtype, torch.float32
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return stitch_block_norms_grad(dy, dx_out, h, x_out, post=post, post_weight=post_weight, post_bias=post_bias,
                                           gate=gate, scale=scale, alpha=alpha, pre=pre, pre_weight=pre_weight,
                                           pre_bias=pre_bias, eps=eps, dx=dx, out=out, workspace=workspace,
                                           tuning=tuning)
    like = h.shape
    rows, cols = _sizes("h", h, 2)
    po, pr = _norm("post", post, post_weight, post_bias), _norm("pre", pre, pre_weight, pre_bias)
    if (dy is None) == (pr != CF_NORM_NONE):
        raise ValueError("dy goes with a norm before the next block (pre \"none\" where only x' was used)")
    gates, vector = _gates(gate, rows), (cols,)
    ph, pxo = _operand("h", h, like, dtype, dev), _operand("x_out", x_out, like, dtype, dev)
    pdy, pdx = _operand("dy", dy, like, dtype, dev), _operand("dx_out", dx_out, like, dtype, dev)
    given = (None,) * 7 if out is None else out
    dh = _made_like("out[0]", given[0], h)
    dx = _made_like("out[1]", given[1], h) if dx else None
    pg = pw = pb = qw = dg = dpw = dpb = dqw = dqb = None
    if gate is not None:
        pg, dg = _operand("gate", gate, (gates, cols), dtype, dev), _made_like("out[2]", given[2], gate)
    if post_weight is not None:
        pw = _operand("post_weight", post_weight, vector, f32, dev)
        dpw = _made_like("out[3]", given[3], post_weight)
    if post_bias is not None:
        pb, dpb = _operand("post_bias", post_bias, vector, f32, dev), _made_like("out[4]", given[4], post_bias)
    if pre_weight is not None:
        qw, dqw = _operand("pre_weight", pre_weight, vector, f32, dev), _made_like("out[5]", given[5], pre_weight)
    if pre_bias is not None:
        _operand("pre_bias", pre_bias, vector, f32, dev)
        dqb = _made_like("out[6]", given[6], pre_bias)
    _launch("cf_stitch_block_norms_grad", (pdy, pdx, ph, pxo, pg, pw, pb, qw, dh.data_ptr(), _at(dx), _at(dg), _at(dpw),
                                           _at(dpb), _at(dqw), _at(dqb), rows, cols, gates, po, pr, scale, alpha, eps, dt),
            dev, workspace, cf_stitch_block_norms_grad_workspace_size, (rows, cols), tuning)
    return dh, dx, dg, dpw, dpb, dqw, dqb


# ---------------------------------------------------------------------------
# log probabilities of given tokens
# ---------------------------------------------------------------------------
def cf_stitch_logprobs(logits, targets, logprob, lse, entropy, top_logprobs, top_ids, rows, vocab, stride, top, scale,
                       dtype, workspace, workspace_bytes, stream=None, tuning=None) -> int:
    L = lib()
    args = (_ptr(logits), _ptr(targets), _ptr(logprob), _ptr(lse), _ptr(entropy), _ptr(top_logprobs), _ptr(top_ids),
            rows, vocab, stride, top, scale, dtype, _ptr(workspace), workspace_bytes, _stream(stream))
    return L.cf_stitch_logprobs(*args) if tuning is None else L.cf_stitch_logprobs_ex(*args, _tun(tuning))


def cf_stitch_logprobs_grad(logits, targets, lse, entropy, dlogprob, dlse, dentropy, dlogits, rows, vocab, stride,
                            dstride, scale, dtype, workspace, workspace_bytes, stream=None, tuning=None) -> int:
    L = lib()
    args = (_ptr(logits), _ptr(targets), _ptr(lse), _ptr(entropy), _ptr(dlogprob), _ptr(dlse), _ptr(dentropy),
            _ptr(dlogits), rows, vocab, stride, dstride, scale, dtype, _ptr(workspace), workspace_bytes,
            _stream(stream))
    return L.cf_stitch_logprobs_grad(*args) if tuning is None else L.cf_stitch_logprobs_grad_ex(*args, _tun(tuning))


def _rows_apart(name, t, shape=None, dtype=None, device=None):
    """(rows, columns, elements from a row to the next) of a matrix whose rows are contiguous, checked."""
    rows, cols = _sizes(name, t, 2)
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if cols > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name} has rows that are not contiguous or that overlap")
    return rows, cols, t.stride(0) if rows > 1 else cols


def stitch_logprobs(logits, targets=None, *, scale=1.0, top=0, entropy=True, out=None, workspace=None, stream=None,
                    tuning=None):
    """(logprob, lse, entropy, top_logprobs, top_ids) of softmax(scale * logits), rows [T, V] of bf16, fp16 or fp32
    that may lie apart (logits[:, :V] of a padded vocabulary): the log probability of each row's target (int64 [T], -1:
    none, 0), log-sum-exp and entropy, all fp32 [T], and the `top` (0..32) largest logits' log probabilities and ids
    [T, top], equal logits by id.  None in the place of what is not asked for.  `out`: five outputs, None for new ones."""
    torch = _torch or _the_torch()
    dt, dev, f32, i64 = _row_dtype("logits", logits), logits.device, torch.float32, torch.int64
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return stitch_logprobs(logits, targets, scale=scale, top=top, entropy=entropy, out=out, workspace=workspace,
                                   tuning=tuning)
    rows, vocab, apart = _rows_apart("logits", logits)
    if not 0 <= top <= min(vocab, 32):
        raise ValueError(f"top is {top}, not in 0..{min(vocab, 32)}")
    if not scale > 0:
        raise ValueError(f"scale is {scale}, not above 0")
    if vocab == 0 and rows > 0:
        raise ValueError("logits have no columns")
    t = _operand("targets", targets, (rows,), i64, dev)
    given = (None,) * 5 if out is None else out
    lse = _made("out[1]", given[1], (rows,), f32, dev)
    logprob = None if targets is None else _made_like("out[0]", given[0], lse)
    h = _made_like("out[2]", given[2], lse) if entropy else None
    tl = _made("out[3]", given[3], (rows, top), f32, dev) if top else None
    ti = _made("out[4]", given[4], (rows, top), i64, dev) if top else None
    _launch("cf_stitch_logprobs", (logits.data_ptr(), t, _at(logprob), lse.data_ptr(), _at(h), _at(tl), _at(ti), rows,
                                   vocab, apart, top, scale, dt), dev, workspace, cf_stitch_workspace_size, (rows, vocab),
            tuning)
    return logprob, lse, h, tl, ti


def stitch_logprobs_grad(logits, targets, lse, dlogprob=None, *, dlse=None, entropy=None, dentropy=None, scale=1.0,
                         out=None, workspace=None, stream=None, tuning=None):
    """The gradient of the logits [T, V] (in their dtype) for the gradients dlogprob, dlse and dentropy (fp32 [T], None:
    0) of stitch_logprobs' results; lse and, with dentropy, entropy are its results: probabilities are off by 2^-24 |lse| of
    themselves, so a row that a mask of the type's lowest number leaves nothing of has no gradient of use.  `out` may be logits, or rows
    apart like theirs, which is up to four times faster than the contiguous one that is made without it where logits' rows
    lie apart and are of no whole 16 bytes."""
    torch = _torch or _the_torch()
    dt, dev, dtype, f32 = _row_dtype("logits", logits), logits.device, logits.dtype, torch.float32
    if _away(dev, stream):
        with _launch_on(dev, stream):
            return stitch_logprobs_grad(logits, targets, lse, dlogprob, dlse=dlse, entropy=entropy, dentropy=dentropy,
                                        scale=scale, out=out, workspace=workspace, tuning=tuning)
    rows, vocab, apart = _rows_apart("logits", logits)
    if not scale > 0:
        raise ValueError(f"scale is {scale}, not above 0")
    if (targets is None) != (dlogprob is None):
        raise ValueError("dlogprob goes with targets")
    if (entropy is None) != (dentropy is None):
        raise ValueError("dentropy goes with entropy")
    if dlogprob is None and dlse is None and dentropy is None:
        raise ValueError("no gradient is given")
    row = (rows,)
    args = (logits.data_ptr(), _operand("targets", targets, row, torch.int64, dev), _operand("lse", lse, row, f32, dev),
            _operand("entropy", entropy, row, f32, dev), _operand("dlogprob", dlogprob, row, f32, dev),
            _operand("dlse", dlse, row, f32, dev), _operand("dentropy", dentropy, row, f32, dev))
    if out is None:
        out, between = torch.empty((rows, vocab), dtype=dtype, device=dev), vocab
    else:
        between = _rows_apart("out", out, (rows, vocab), dtype, dev)[2]
    _launch("cf_stitch_logprobs_grad", (*args, out.data_ptr(), rows, vocab, apart, between, scale, dt), dev, workspace,
            cf_stitch_workspace_size, (rows, vocab), tuning)
    return out
