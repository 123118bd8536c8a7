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
