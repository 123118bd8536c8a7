"""Plain, slow, fp64 CPU oracle for the fused GEMM + row-reduce/broadcast path.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or
execute this module: only ``tests/``, ``__graft_entry__.smoke()`` and the
``cpu_baseline`` / ``--impl reference`` legs of ``bench.py`` use it.  It shares
no code with the CUDA path; the only thing both sides share is the seeded
input generator, which holds none of the method's arithmetic.

What is computed, and where it is defined
-----------------------------------------
The pages describe *exact* fusion: the fused kernel must reach the result of
the unfused operator chain (the fusion keeps the semantics of the unfused
operators: ComFuse, Fusion Spec IR, Eq. (10); ownership legality: sass2mlir
"Kernel fusion", section "Epilogue fusion - the core technique").  So the oracle is the unfused chain
written out in float64 on the same (bf16 / fp32) input values:

* MatMul      P = X . W                       (ComFuse, Eq. (6) notation)
* Stage 1     x = alpha * P + bias            (ComFuse, Stage-Stream Execution
                                               Model, Fig. 3: x = alpha*Acc+Bias)
* activation  g = GELU_tanh(x) or g = x       (a unary compute node, ComFuse,
                                               Fusion Spec IR mapping Phi)
* reduction   LayerNorm / RMSNorm / Softmax as "reduce over the inputs,
              normalise the original values" (ComFuse, nested Fusion Spec IR
              at reductions, which names all three patterns)
* stitched    y = A^3 + b[row]; rowwise softmax (AStitch, "Adaptive thread
              mapping": row reductions on 750000x32 and 64x30000)

Pages cited (full titles):
  ComFuse  -- "ComFuse: Fusing Complex Memory-Intensive Subgraphs with
              Compute-Intensive Kernels For Modern GPU Architectures"
  AStitch  -- "AStitch: enabling a new multi-dimensional optimization space for
              memory-intensive ML training and inference on modern SIMT
              architectures"
  sass2mlir -- the sass2mlir "kernel fusion" page ("Two answers to the same
              idle GPU": CUDA graphs, then "How we fuse kernels")

Readings taken where the pages are silent:
  * LayerNorm variance is the biased one (divide by N), eps inside the square
    root, gamma/beta applied after normalising; with GELU the norm is taken
    over the post-GELU values.
  * RMSNorm divides each value by sqrt(mean of the squares + eps) with no mean
    subtraction (the usual definition, Zhang & Sennrich 2019); gamma scales
    after normalising and beta, when given, is added last.
  * Residual add + norm: the residual R is added after the activation node
    and before the reduction (the "add & norm" of a transformer block).
  * B2BGEMM: O = S . W2 with S = F(alpha * X.W1 + b1) held in bf16 -- the
    dtype of the intermediate tensor the unfused chain would materialise
    (the tensor cores consume bf16 operands); F is GELU(tanh), the row
    softmax over N1 or the row LayerNorm over N1 (gamma1, beta1 per column).
  * Masked softmax: a causal mask keeps element (i, j) of the scaled scores
    iff j <= i + offset (masked elements are -inf before the softmax); a row
    with no kept element is all zeros.
  * Softmax scale multiplies the accumulator before max/exp; an optional bias
    is added after scaling.  Exponent base e.
  * GELU is the tanh form: 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))).
  * pow(A, 3) is the real cube with its sign (A*A*A).
  * Stitched add + LayerNorm: x = A + R (R optional), LayerNorm over each
    row as above, gamma/beta indexed by column.
  * Stitched power -> broadcast -> add -> softmax: y = A + w[col]^p with w > 0
    (the real power function w^p = exp(p ln w)), then the row softmax; the
    power of each column is a one-to-many value (AStitch's power -> broadcast
    -> add example, "What people did before").
  * Stitched BatchNorm (training-mode statistics): per column j the mean and
    the biased variance over all rows; y = (A - mean_j) / sqrt(var_j + eps)
    * gamma_j + beta_j.  The column statistic is a one-to-many dependency
    over every row (AStitch, "Four stitching schemes": Regional when one
    block holds all rows of its columns, Global otherwise).

Every function here is pinned by ``tests/test_oracle_pins.py`` against closed
forms, invariants, brute force on tiny inputs and library routines.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = [
    "activation",
    "activation_slope",
    "gemm_linear",
    "gemm_linear_grad",
    "norm_rows",
    "block_norms",
    "block_norms_grad",
    "logprobs",
    "logprobs_grad",
    "gelu_tanh_slope",
    "grouped_gemm",
    "grouped_gemm_dgrad",
    "grouped_gemm_wgrad",
    "gemm_lora",
    "gemm",
    "gemm_naive",
    "gelu_tanh",
    "layernorm_rows",
    "rmsnorm_rows",
    "softmax_rows",
    "gemm_bias_rownorm",
    "gemm_bias_rmsnorm",
    "gemm_bias_residual_norm",
    "gemm_rowsoftmax_causal",
    "b2b_gemm",
    "stitch_add_layernorm",
    "stitch_batchnorm",
    "gemm_rowsoftmax",
    "stitch_rowreduce_broadcast",
    "stitch_powadd_softmax",
    "ROW_CHUNK",
]

# Row chunk used to bound the oracle's memory on the large configurations.
# Chunking over rows changes nothing: every row is computed independently.
ROW_CHUNK = 1024

_SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)
_GELU_CUBIC = 0.044715


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def gemm(X, W) -> np.ndarray:
    """P = X . W in float64 (ComFuse, Eq. (6): X in R^{MxK}, W in R^{KxN}).

    bf16 inputs widen exactly to float64 and every bf16 x bf16 product is
    exact in float64, so the only rounding is the float64 summation.
    """
    X = _f64(X)
    W = _f64(W)
    if X.ndim != 2 or W.ndim != 2 or X.shape[1] != W.shape[0]:
        raise ValueError(f"gemm: incompatible shapes {X.shape} x {W.shape}")
    return X @ W


def gemm_naive(X, W) -> np.ndarray:
    """Triple-loop MatMul, pure Python.  For tiny inputs only (pins gemm)."""
    X = _f64(X)
    W = _f64(W)
    M, K = X.shape
    K2, N = W.shape
    if K != K2:
        raise ValueError("gemm_naive: inner dimensions differ")
    P = np.zeros((M, N), dtype=np.float64)
    for i in range(M):
        for j in range(N):
            s = 0.0
            for k in range(K):
                s += float(X[i, k]) * float(W[k, j])
            P[i, j] = s
    return P


def gelu_tanh(x) -> np.ndarray:
    """GELU, tanh form: 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))."""
    x = _f64(x)
    return 0.5 * x * (1.0 + np.tanh(_SQRT_2_OVER_PI * (x + _GELU_CUBIC * x * x * x)))


def layernorm_rows(g, gamma, beta, eps: float) -> np.ndarray:
    """LayerNorm over the last axis, two-pass.

    mean = (1/N) sum g;  var = (1/N) sum (g - mean)^2  (biased);
    y = (g - mean) / sqrt(var + eps) * gamma + beta.
    This is the pattern the ComFuse Fusion Spec IR nests at a Reduction
    node -- reduce over the inputs, then normalise the original values: the first
    reduction (mean) feeds the second (variance), whose statistic is then
    broadcast back over the row together with the bypassed values.
    """
    g = _f64(g)
    mean = g.mean(axis=-1, keepdims=True)
    d = g - mean
    var = (d * d).mean(axis=-1, keepdims=True)
    return d / np.sqrt(var + float(eps)) * _f64(gamma) + _f64(beta)


def rmsnorm_rows(g, gamma, beta, eps: float) -> np.ndarray:
    """y = g / sqrt(mean(g^2) + eps) * gamma (+ beta), each row of g.

    RMSNorm as a nested stage DAG (ComFuse, Fusion Spec IR): the reduction is
    the mean of the squares over the row; the PostOp rescales the original
    values.  ``beta`` may be None (no shift node).
    """
    g = _f64(g)
    ms = (g * g).mean(axis=-1, keepdims=True)
    y = g / np.sqrt(ms + float(eps)) * _f64(gamma)
    return y if beta is None else y + _f64(beta)


def softmax_rows(z) -> np.ndarray:
    """Row softmax: m = max z; e = exp(z - m); y = e / sum(e)."""
    z = _f64(z)
    m = z.max(axis=-1, keepdims=True)
    e = np.exp(z - m)
    return e / e.sum(axis=-1, keepdims=True)


def _row_chunks(M: int, rows):
    if rows is None:
        for r0 in range(0, M, ROW_CHUNK):
            yield np.arange(r0, min(M, r0 + ROW_CHUNK))
    else:
        rows = np.asarray(rows, dtype=np.int64)
        for r0 in range(0, rows.size, ROW_CHUNK):
            yield rows[r0:r0 + ROW_CHUNK]


def gemm_bias_rownorm(X, W, bias, gamma, beta, *, alpha: float = 1.0,
                      eps: float = 1e-5, act: str = "none", rows=None) -> np.ndarray:
    """y = LayerNorm(act(alpha * X.W + bias)) * gamma + beta, row by row.

    ComFuse, Stage-Stream Execution Model, Fig. 3 (stage 1: x = alpha*Acc+Bias,
    mean; stage 2: x - mean, ...) with an optional GELU node between the
    bias add and the reductions.  ``rows`` selects a subset of output rows
    (every row is independent, so a sampled row is exact).
    ``bias`` may be None (no bias node).
    """
    if act not in ("none", "gelu_tanh"):
        raise ValueError(f"unknown activation {act!r}")
    X = np.asarray(X)
    M = X.shape[0]
    N = np.asarray(W).shape[1]
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    b = np.zeros(N) if bias is None else _f64(bias)
    o = 0
    for idx in _row_chunks(M, rows):
        x = float(alpha) * gemm(X[idx], W) + b
        g = gelu_tanh(x) if act == "gelu_tanh" else x
        out[o:o + idx.size] = layernorm_rows(g, gamma, beta, eps)
        o += idx.size
    return out


def gemm_bias_rmsnorm(X, W, bias, gamma, beta=None, *, alpha: float = 1.0,
                      eps: float = 1e-5, act: str = "none", rows=None) -> np.ndarray:
    """y = RMSNorm(act(alpha * X.W + bias)) * gamma (+ beta), row by row.

    The same stage-1 nodes as ``gemm_bias_rownorm`` (ComFuse, Stage-Stream
    Execution Model, Fig. 3: x = alpha*Acc+Bias, then the optional GELU node)
    followed by the RMSNorm reduction and PostOp.
    """
    if act not in ("none", "gelu_tanh"):
        raise ValueError(f"unknown activation {act!r}")
    X = np.asarray(X)
    M = X.shape[0]
    N = np.asarray(W).shape[1]
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    b = np.zeros(N) if bias is None else _f64(bias)
    o = 0
    for idx in _row_chunks(M, rows):
        x = float(alpha) * gemm(X[idx], W) + b
        g = gelu_tanh(x) if act == "gelu_tanh" else x
        out[o:o + idx.size] = rmsnorm_rows(g, gamma, beta, eps)
        o += idx.size
    return out


def gemm_bias_residual_norm(X, W, bias, R, gamma, beta, *, alpha: float = 1.0, eps: float = 1e-5,
                            act: str = "none", norm: str = "layer", rows=None) -> np.ndarray:
    """y = Norm(act(alpha * X.W + bias) + R) * gamma (+ beta), row by row.

    sass2mlir, "Epilogue fusion - the core technique": activation, norm and
    residual add run on the accumulator in the producer's epilogue.  The
    residual R [M, N] is one more elementwise node before the reduction
    (ComFuse, Stage-Stream Execution Model: stage-1 nodes, then the row
    reduction).  norm is "layer" (LayerNorm) or "rms" (RMSNorm; beta may be
    None there).
    """
    if act not in ("none", "gelu_tanh"):
        raise ValueError(f"unknown activation {act!r}")
    if norm not in ("layer", "rms"):
        raise ValueError(f"unknown norm {norm!r}")
    X = np.asarray(X)
    R = np.asarray(R)
    M = X.shape[0]
    N = np.asarray(W).shape[1]
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    b = np.zeros(N) if bias is None else _f64(bias)
    o = 0
    for idx in _row_chunks(M, rows):
        x = float(alpha) * gemm(X[idx], W) + b
        g = (gelu_tanh(x) if act == "gelu_tanh" else x) + _f64(R[idx])
        out[o:o + idx.size] = (layernorm_rows(g, gamma, beta, eps) if norm == "layer"
                               else rmsnorm_rows(g, gamma, beta, eps))
        o += idx.size
    return out


def gemm_rowsoftmax(X, W, *, scale: float, bias=None, rows=None) -> np.ndarray:
    """y = softmax(scale * X.W (+ bias)) over each row."""
    X = np.asarray(X)
    M = X.shape[0]
    N = np.asarray(W).shape[1]
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    o = 0
    for idx in _row_chunks(M, rows):
        z = float(scale) * gemm(X[idx], W)
        if bias is not None:
            z = z + _f64(bias)
        out[o:o + idx.size] = softmax_rows(z)
        o += idx.size
    return out


def gemm_rowsoftmax_causal(X, W, *, scale: float, offset: int, bias=None, rows=None) -> np.ndarray:
    """y = softmax(mask(scale * X.W (+ bias))) over each row, where the mask
    keeps column j of row i iff j <= i + offset; a fully masked row is 0.

    A masked reduction node ahead of Softmax's nested stage DAG (ComFuse,
    Fusion Spec IR): masked elements take no part in the max or the sum and
    are 0 in the output.
    """
    X = np.asarray(X)
    M = X.shape[0]
    N = np.asarray(W).shape[1]
    idx_all = np.arange(M) if rows is None else np.asarray(rows)
    out = np.zeros((idx_all.size, N), dtype=np.float64)
    o = 0
    for idx in _row_chunks(M, rows):
        z = float(scale) * gemm(X[idx], W)
        if bias is not None:
            z = z + _f64(bias)
        keep = np.arange(N)[None, :] <= (idx[:, None] + int(offset))
        for r in range(idx.size):
            if keep[r].any():
                out[o + r, keep[r]] = softmax_rows(z[r, keep[r]][None, :])[0]
        o += idx.size
    return out


def b2b_gemm(X, W1, W2, *, op: str, alpha: float = 1.0, b1=None, rows=None, gamma1=None, beta1=None,
             eps: float = 1e-5) -> np.ndarray:
    """O = bf16(F(alpha * X.W1 + b1)) . W2, F = GELU_tanh, the row softmax or
    the row LayerNorm (with gamma1, beta1 over the N1 columns).

    ComFuse, B2BGEMM (Eqs. 3-7): MatMul_1, the epilogue F giving S_tile
    (Eq. 3), MatMul_2 over the intermediate dimension N1 (Eqs. 4-5).  The
    intermediate S is rounded to bf16 (round to nearest even), the precision
    of the tensor the unfused chain stores between the two GEMMs.
    """
    if op not in ("softmax", "gelu_tanh", "layernorm"):
        raise ValueError(f"unknown op {op!r}")
    X = np.asarray(X)
    M = X.shape[0]
    N2 = np.asarray(W2).shape[1]
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N2), dtype=np.float64)
    b = 0.0 if b1 is None else _f64(b1)
    o = 0
    for idx in _row_chunks(M, rows):
        z = float(alpha) * gemm(X[idx], W1) + b
        if op == "softmax":
            S = softmax_rows(z)
        elif op == "gelu_tanh":
            S = gelu_tanh(z)
        else:
            S = layernorm_rows(z, gamma1, beta1, eps)
        S = _round_bf16(S)
        out[o:o + idx.size] = gemm(S, W2)
        o += idx.size
    return out


def _round_bf16(a) -> np.ndarray:
    """Nearest bf16 value (ties to even) of each element, via float32."""
    f = np.asarray(a, dtype=np.float64).astype(np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32).astype(np.float64)


def stitch_add_layernorm(A, R, gamma, beta, eps: float, rows=None) -> np.ndarray:
    """out = LayerNorm(A + R) * gamma + beta over each row (R may be None).

    AStitch, "Four stitching schemes": an elementwise producer (Local), two
    reductions over the row (mean, then the variance around it) and their
    broadcast back, with column parameters shared by every row (a
    one-to-many dependency: Regional).
    """
    A = np.asarray(A)
    M, N = A.shape
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    o = 0
    for idx in _row_chunks(M, rows):
        x = _f64(A[idx])
        if R is not None:
            x = x + _f64(np.asarray(R)[idx])
        out[o:o + idx.size] = layernorm_rows(x, gamma, beta, eps)
        o += idx.size
    return out


def stitch_batchnorm(A, gamma, beta, eps: float):
    """BatchNorm over the rows of A [rows, cols] with batch statistics.

    mean_j = (1/rows) sum_i A_ij;  var_j = (1/rows) sum_i (A_ij - mean_j)^2;
    out_ij = (A_ij - mean_j) / sqrt(var_j + eps) * gamma_j + beta_j.
    Returns (out, mean, var).  Every output depends on every row of its
    column: the reduction runs along the other axis from the row reductions
    (AStitch, "Four stitching schemes", column reduction -> broadcast).
    """
    A = _f64(A)
    mean = A.mean(axis=0)
    d = A - mean
    var = (d * d).mean(axis=0)
    return d / np.sqrt(var + float(eps)) * _f64(gamma) + _f64(beta), mean, var


def stitch_rowreduce_broadcast(A, row_bias, rows=None) -> np.ndarray:
    """Stitched memory-intensive subgraph (AStitch, "Adaptive thread mapping"):

    y = A*A*A + b[row]  (elementwise power, then a broadcast row bias);
    m = rowmax(y); s = rowsum(exp(y - m)); out = exp(y - m) / s.
    """
    A = np.asarray(A)
    b = np.asarray(row_bias)
    M, N = A.shape
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    o = 0
    for idx in _row_chunks(M, rows):
        a = _f64(A[idx])
        y = a * a * a + _f64(b[idx])[:, None]
        out[o:o + idx.size] = softmax_rows(y)
        o += idx.size
    return out


def stitch_powadd_softmax(A, w, p: float, rows=None) -> np.ndarray:
    """Stitched subgraph with both one-to-many dependencies (AStitch, "What
    people did before": an expensive element-wise power feeding a broadcast
    and an add; "Four stitching schemes": the reduction feeding consumers):

    y = A + w[col] ** p   (w > 0: the real power w^p = exp(p ln w));
    m = rowmax(y); s = rowsum(exp(y - m)); out = exp(y - m) / s.
    """
    A = np.asarray(A)
    w = _f64(w)
    if np.any(w <= 0):
        raise ValueError("stitch_powadd_softmax: w must be positive")
    pw = w ** float(p)
    M, N = A.shape
    out_rows = M if rows is None else len(rows)
    out = np.empty((out_rows, N), dtype=np.float64)
    o = 0
    for idx in _row_chunks(M, rows):
        y = _f64(A[idx]) + pw[None, :]
        out[o:o + idx.size] = softmax_rows(y)
        o += idx.size
    return out


def gelu_tanh_slope(x) -> np.ndarray:
    """d/dx of gelu_tanh: (1 + t)/2 + x (1 - t^2)/2 * s (1 + 3*0.044715 x^2), t = tanh(s (x + 0.044715 x^3))."""
    x = _f64(x)
    s = math.sqrt(2.0 / math.pi)
    t = np.tanh(s * (x + 0.044715 * x ** 3))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * s * (1.0 + 3.0 * 0.044715 * x * x)


def grouped_gemm(X, W, offsets, *, act: str = "none"):
    """(Y, Z): for the rows r in [offsets[e], offsets[e+1]), Z[r] = X[r].W[e] and Y[r] = act(Z[r]).

    Rows of no group are zero in both."""
    X, W = _f64(X), _f64(W)
    Z = np.zeros((X.shape[0], W.shape[2]))
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        Z[lo:hi] = X[lo:hi] @ W[e]
    return (gelu_tanh(Z) if act == "gelu_tanh" else Z.copy()), Z


def grouped_gemm_dgrad(dY, W, offsets, *, preact=None) -> np.ndarray:
    """dX[r] = (dY[r].W[e]^T) * gelu_tanh'(preact[r]) for the rows of each group; rows of no group are zero."""
    dY, W = _f64(dY), _f64(W)
    dX = np.zeros((dY.shape[0], W.shape[1]))
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        dX[lo:hi] = dY[lo:hi] @ W[e].T
        if preact is not None:
            dX[lo:hi] *= gelu_tanh_slope(preact[lo:hi])
    return dX


def grouped_gemm_wgrad(X, dY, offsets) -> np.ndarray:
    """dW[e] = X[rows of e]^T.dY[rows of e]; zero for an empty group."""
    X, dY = _f64(X), _f64(dY)
    return np.stack([X[int(lo):int(hi)].T @ dY[int(lo):int(hi)] for lo, hi in zip(offsets[:-1], offsets[1:])])


def gemm_lora(X, W, bias, A, B, offsets, adapters, scale=None) -> np.ndarray:
    """Y[r] = X[r].W + bias + scale[a] (X[r].A[a]).B[a], a the adapter of the row's request (-1: none).

    Rows of no request are zero."""
    X, W = _f64(X), _f64(W)
    Y = np.zeros((X.shape[0], W.shape[1]))
    for s in range(len(adapters)):
        lo, hi, a = int(offsets[s]), int(offsets[s + 1]), int(adapters[s])
        Y[lo:hi] = X[lo:hi] @ W + (0.0 if bias is None else _f64(bias))
        if a >= 0:
            Y[lo:hi] += (1.0 if scale is None else float(scale[a])) * ((X[lo:hi] @ _f64(A[a])) @ _f64(B[a]))
    return Y


# ---------------------------------------------------------------------------
# dense layer
# ---------------------------------------------------------------------------
def _logistic(z) -> np.ndarray:
    return 0.5 * (1.0 + np.tanh(0.5 * _f64(z)))


def activation(act: str, z) -> np.ndarray:
    z = _f64(z)
    if act == "gelu_tanh":
        return gelu_tanh(z)
    if act == "silu":
        return z * _logistic(z)
    return np.where(z > 0.0, z, 0.0) if act == "relu" else z.copy()


def activation_slope(act: str, z) -> np.ndarray:
    """d/dz of it; the slope of ReLU at 0 is 0."""
    z = _f64(z)
    if act == "gelu_tanh":
        return gelu_tanh_slope(z)
    if act == "silu":
        p = _logistic(z)
        return p * (1.0 + z * (1.0 - p))
    return (z > 0.0).astype(np.float64) if act == "relu" else np.ones_like(z)


def gemm_linear(X, W, bias=None, *, act: str = "none", residual=None):
    """(Y, Z) with Z = X.W + bias and Y = act(Z) + residual."""
    Z = _f64(X) @ _f64(W) + (0.0 if bias is None else _f64(bias))
    return activation(act, Z) + (0.0 if residual is None else _f64(residual)), Z


def gemm_linear_grad(dY, X, W, *, act: str = "none", preact=None):
    """(dX, dW, dbias): dZ = dY act'(Z), dX = dZ.W^T, dW = X^T.dZ, dbias = sum over the rows of dZ."""
    dZ = _f64(dY) if act == "none" else _f64(dY) * activation_slope(act, preact)
    return dZ @ _f64(W).T, _f64(X).T @ dZ, dZ.sum(0)


# ---------------------------------------------------------------------------
# norms before and after a block
# ---------------------------------------------------------------------------
def norm_rows(kind: str, t, eps: float):
    """(normalised rows, 1 / what they were divided by); kind "none", "rms" or "layer"."""
    t = _f64(t)
    if kind == "none":
        return t, np.ones((t.shape[0], 1))
    c = t - t.mean(1, keepdims=True) if kind == "layer" else t
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + float(eps))
    return c * r, r


def _gate_rows(gate, rows: int):
    return 1.0 if gate is None else np.repeat(_f64(gate), rows // len(gate), axis=0)


def _affine(t, weight, bias):
    return t * (1.0 if weight is None else _f64(weight)) + (0.0 if bias is None else _f64(bias))


def block_norms(h, x, *, post="none", post_weight=None, post_bias=None, gate=None, scale=1.0, alpha=1.0, pre="none",
                pre_weight=None, pre_bias=None, eps: float = 1e-5):
    """(x', y): x' = alpha x + scale gate Post(h), y = Pre(x'); x may be None (0); gate [G, N], G a divisor of the
    rows, which share a gate in equal runs."""
    h = _f64(h)
    p = _affine(norm_rows(post, h, eps)[0], post_weight, post_bias)
    out = float(scale) * _gate_rows(gate, len(h)) * p + (0.0 if x is None else float(alpha) * _f64(x))
    return out, _affine(norm_rows(pre, out, eps)[0], pre_weight, pre_bias)


def _norm_grad(kind: str, hat, r, g):
    if kind == "none":
        return g
    d = g - hat * (g * hat).mean(1, keepdims=True)
    return r * (d - g.mean(1, keepdims=True) if kind == "layer" else d)


def block_norms_grad(dy, dx_out, h, x_out, *, post="none", post_weight=None, post_bias=None, gate=None, scale=1.0,
                     alpha=1.0, pre="none", pre_weight=None, eps: float = 1e-5) -> dict:
    """Gradients of block_norms for the gradients dy of y and dx_out of x' (either may be None): h, x, gate,
    post_weight, post_bias, pre_weight, pre_bias."""
    h, xo = _f64(h), _f64(x_out)
    rows = len(h)
    dx = np.zeros_like(xo) if dx_out is None else _f64(dx_out).copy()
    out = {}
    if dy is not None:
        hat, r = norm_rows(pre, xo, eps)
        out["pre_weight"], out["pre_bias"] = (_f64(dy) * hat).sum(0), _f64(dy).sum(0)
        dx += _norm_grad(pre, hat, r, _f64(dy) * (1.0 if pre_weight is None else _f64(pre_weight)))
    out["x"] = float(alpha) * dx
    hat, r = norm_rows(post, h, eps)
    dp = float(scale) * dx
    if gate is not None:
        out["gate"] = (dp * _affine(hat, post_weight, post_bias)).reshape(len(gate), -1, h.shape[1]).sum(1)
    dp = dp * _gate_rows(gate, rows)
    out["post_weight"], out["post_bias"] = (dp * hat).sum(0), dp.sum(0)
    out["h"] = _norm_grad(post, hat, r, dp * (1.0 if post_weight is None else _f64(post_weight)))
    return out


# ---------------------------------------------------------------------------
# log probabilities of given tokens
# ---------------------------------------------------------------------------
def logprobs(logits, targets=None, *, scale: float = 1.0, top: int = 0):
    """dict of logprob, lse, entropy, top_logprobs, top_ids of softmax(scale logits).

    A target of -1 has logprob 0.  A row of nothing but -inf has lse and logprob -inf and entropy 0; one with a NaN or
    +inf has NaNs.  The top ids are by logit, equal ones by id; a NaN counts as the largest."""
    raw = _f64(logits)
    z = raw * float(scale)
    rows = np.arange(len(z))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = z.max(1, keepdims=True)
        bad = ~(m < np.inf)[:, 0]
        none = (m == -np.inf)[:, 0]
        d = z - np.where(none[:, None], 0.0, m)
        e = np.exp(d)
        s = e.sum(1)
        lse = np.where(none, -np.inf, m[:, 0] + np.log(s))
        entropy = np.where(none, 0.0, np.log(s) - (e * np.where(e > 0, d, 0.0)).sum(1) / s)
        logp = np.where(none[:, None], -np.inf, d - np.log(s)[:, None])
    lse, entropy = (np.where(bad, np.nan, v) for v in (lse, entropy))
    logp[bad] = np.nan
    out = {"lse": lse, "entropy": entropy}
    if targets is not None:
        t = np.asarray(targets)
        out["logprob"] = np.where(t < 0, 0.0, logp[rows, np.maximum(t, 0)])
    if top > 0:
        order = np.argsort(-np.where(np.isnan(raw), np.inf, raw), axis=1, kind="stable")
        first = np.argsort(~np.isnan(np.take_along_axis(raw, order, 1)), axis=1, kind="stable")  # NaN before inf
        ids = np.take_along_axis(order, first, 1)[:, :top]
        out["top_ids"], out["top_logprobs"] = ids, np.take_along_axis(logp, ids, 1)
    return out


def logprobs_grad(logits, targets=None, *, dlogprob=None, dlse=None, dentropy=None, scale: float = 1.0,
                  lse=None, entropy=None) -> np.ndarray:
    """The gradient of the logits; lse and entropy may be given (those of `logprobs` otherwise).  A row of nothing but
    -inf has none."""
    raw = _f64(logits)
    f = logprobs(raw, scale=scale)
    lse = f["lse"] if lse is None else _f64(lse)
    entropy = f["entropy"] if entropy is None else _f64(entropy)
    zero = np.zeros(len(raw))
    dlp = zero if dlogprob is None or targets is None else np.where(np.asarray(targets) < 0, 0.0, _f64(dlogprob))
    dl, dh = (zero if v is None else _f64(v) for v in (dlse, dentropy))
    none = np.all(raw == -np.inf, axis=1)
    with np.errstate(invalid="ignore"):
        logp = raw * float(scale) - np.where(none, 0.0, lse)[:, None]
        p = np.exp(logp)
        d = p * ((dl - dlp)[:, None] - dh[:, None] * (np.where(p > 0, logp, 0.0) + entropy[:, None]))
    if targets is not None:
        t = np.asarray(targets)
        d[np.arange(len(raw)), np.maximum(t, 0)] += dlp
    d[none] = 0.0
    return d * float(scale)
