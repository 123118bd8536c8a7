"""The oracle's grouped products and low-rank adapters against triple loops
in exact rational arithmetic and against differences of the scalar loss they
are the gradients of (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

import oracle

OFFSETS = [1, 3, 3, 7]  # a row of no group before and behind, an empty group
T, K, N, E = 9, 3, 4, 3


def _ints(*shape, seed):
    return np.random.Generator(np.random.PCG64(seed)).integers(-4, 5, size=shape).astype(np.float64)


def _group(r):
    return next((e for e in range(E) if OFFSETS[e] <= r < OFFSETS[e + 1]), None)


def test_grouped_gemm_is_the_triple_loop():
    X, W = _ints(T, K, seed=1), _ints(E, K, N, seed=2)
    Y, Z = oracle.grouped_gemm(X, W, OFFSETS)
    for r in range(T):
        e = _group(r)
        for n in range(N):
            want = 0 if e is None else sum(Fraction(X[r, k]) * Fraction(W[e, k, n]) for k in range(K))
            assert Y[r, n] == want and Z[r, n] == want
    Y, Z = oracle.grouped_gemm(X, W, OFFSETS, act="gelu_tanh")
    assert np.array_equal(Y, oracle.gelu_tanh(Z))


def test_gradients_are_the_differences_of_the_loss():
    """loss = sum(G * gelu(X W1) W2): dgrad through the activation, wgrad of both layers."""
    rng = np.random.Generator(np.random.PCG64(3))
    X, W1, W2 = rng.standard_normal((T, K)), rng.standard_normal((E, K, N)), rng.standard_normal((E, N, 2))
    G = rng.standard_normal((T, 2))

    def loss(x, w1, w2):
        h, _ = oracle.grouped_gemm(x, w1, OFFSETS, act="gelu_tanh")
        return float((G * oracle.grouped_gemm(h, w2, OFFSETS)[0]).sum())

    H, Z = oracle.grouped_gemm(X, W1, OFFSETS, act="gelu_tanh")
    dZ = oracle.grouped_gemm_dgrad(G, W2, OFFSETS, preact=Z)
    grads = [oracle.grouped_gemm_dgrad(dZ, W1, OFFSETS), oracle.grouped_gemm_wgrad(X, dZ, OFFSETS),
             oracle.grouped_gemm_wgrad(H, G, OFFSETS)]
    args = [X, W1, W2]
    h = 1e-5
    for i, (g, a) in enumerate(zip(grads, args)):
        assert g.shape == a.shape
        for at in np.ndindex(a.shape):
            hi, lo = [v.copy() for v in args], [v.copy() for v in args]
            hi[i][at] += h
            lo[i][at] -= h
            # central differences: O(h^2) truncation plus cancellation of about 1e-16 / h
            assert abs((loss(*hi) - loss(*lo)) / (2 * h) - g[at]) < 1e-8, (i, at)
    assert not grads[1][1].any() and not grads[2][1].any()  # the empty group


@pytest.mark.parametrize("scale", [None, [2.0, -3.0]])
def test_lora_is_the_triple_loop(scale):
    X, W, A, B = _ints(T, K, seed=4), _ints(K, N, seed=5), _ints(2, K, 2, seed=6), _ints(2, 2, N, seed=7)
    bias, adapters = _ints(N, seed=8), [1, 0, -1]
    Y = oracle.gemm_lora(X, W, bias, A, B, OFFSETS, adapters, scale)
    for r in range(T):
        s = _group(r)
        for n in range(N):
            want = Fraction(0)
            if s is not None:
                want = sum(Fraction(X[r, k]) * Fraction(W[k, n]) for k in range(K)) + Fraction(bias[n])
                a = adapters[s]
                if a >= 0:
                    low = [sum(Fraction(X[r, k]) * Fraction(A[a, k, j]) for k in range(K)) for j in range(2)]
                    f = Fraction(1) if scale is None else Fraction(scale[a])
                    want += f * sum(low[j] * Fraction(B[a, j, n]) for j in range(2))
            assert Y[r, n] == want


def test_mistakes_show():
    """What the loops above would catch: the neighbour's weights, a group's last row lost, the adapter's scale."""
    X, W = _ints(T, K, seed=1), _ints(E, K, N, seed=2)
    right = oracle.grouped_gemm(X, W, OFFSETS)[0]
    assert not np.array_equal(right, oracle.grouped_gemm(X, W[::-1], OFFSETS)[0])
    assert not np.array_equal(right, oracle.grouped_gemm(X, W, [1, 3, 3, 6])[0])
    A, B = _ints(2, K, 2, seed=6), _ints(2, 2, N, seed=7)
    one = oracle.gemm_lora(X, W[0], None, A, B, OFFSETS, [1, 0, -1], [1.0, 1.0])
    assert not np.array_equal(one, oracle.gemm_lora(X, W[0], None, A, B, OFFSETS, [1, 0, -1], [1.0, 2.0]))
