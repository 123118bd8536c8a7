"""The oracle's dense layer, norms around a block and log probabilities against
plain loops and against differences of the scalar loss whose gradient they
give (CPU)."""
import itertools
import math

import numpy as np
import pytest

import oracle


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _differences(loss, args, grads, h=1e-5, tol=2e-8):
    """Central differences of loss in every element of args[k] against grads[k]: O(h^2) truncation (third
    derivatives of order one) plus cancellation of about 1e-15 / h."""
    for k, g in grads.items():
        a = args[k]
        assert g.shape == a.shape, k
        for at in np.ndindex(a.shape):
            hi, lo = dict(args), dict(args)
            hi[k], lo[k] = a.copy(), a.copy()
            hi[k][at] += h
            lo[k][at] -= h
            assert abs((loss(**hi) - loss(**lo)) / (2 * h) - g[at]) < tol, (k, at)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu", "relu"])
def test_linear(act):
    r = _rng(1)
    a = dict(X=r.standard_normal((3, 4)), W=r.standard_normal((4, 5)), bias=r.standard_normal(5),
             R=r.standard_normal((3, 5)))
    G = r.standard_normal((3, 5))
    Y, Z = oracle.gemm_linear(a["X"], a["W"], a["bias"], act=act, residual=a["R"])
    f = {"none": lambda z: z, "relu": lambda z: max(z, 0.0), "silu": lambda z: z / (1 + math.exp(-z)),
         "gelu_tanh": lambda z: 0.5 * z * (1 + math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}[act]
    for i, j in itertools.product(range(3), range(5)):
        z = sum(a["X"][i, k] * a["W"][k, j] for k in range(4)) + a["bias"][j]
        assert abs(Z[i, j] - z) < 1e-13 and abs(Y[i, j] - f(z) - a["R"][i, j]) < 1e-13
    dX, dW, db = oracle.gemm_linear_grad(G, a["X"], a["W"], act=act, preact=Z)

    def loss(X, W, bias, R):
        return float((G * oracle.gemm_linear(X, W, bias, act=act, residual=R)[0]).sum())

    _differences(loss, a, dict(X=dX, W=dW, bias=db, R=G))


@pytest.mark.parametrize("post,pre,gates", [("rms", "rms", 2), ("layer", "layer", 1), ("none", "rms", 6),
                                            ("layer", "none", 3), ("rms", "layer", 0)])
def test_block_norms(post, pre, gates):
    r = _rng(2)
    T, N, scale, alpha, eps = 6, 5, 0.7, 1.3, 1e-3
    a = dict(h=r.standard_normal((T, N)), x=r.standard_normal((T, N)), post_weight=r.standard_normal(N),
             post_bias=r.standard_normal(N), pre_weight=r.standard_normal(N), pre_bias=r.standard_normal(N))
    if gates:
        a["gate"] = r.standard_normal((gates, N))
    kw = dict(post=post, pre=pre, scale=scale, alpha=alpha, eps=eps)
    G, GX = r.standard_normal((T, N)), r.standard_normal((T, N))
    xo, y = oracle.block_norms(**a, **kw)
    for t in range(T):  # one row by hand
        h = a["h"][t]
        c = h - h.mean() if post == "layer" else h
        p = (c / math.sqrt((c * c).sum() / N + eps) if post != "none" else h) * a["post_weight"] + a["post_bias"]
        g = a["gate"][t // (T // gates)] if gates else 1.0
        want = alpha * a["x"][t] + scale * g * p
        assert np.abs(xo[t] - want).max() < 1e-13
        c = want - want.mean() if pre == "layer" else want
        want = (c / math.sqrt((c * c).sum() / N + eps) if pre != "none" else c) * a["pre_weight"] + a["pre_bias"]
        assert np.abs(y[t] - want).max() < 1e-13

    def loss(**v):
        xo, y = oracle.block_norms(**v, **kw)
        return float((G * y).sum() + (GX * xo).sum())

    g = oracle.block_norms_grad(G, GX, a["h"], xo, post_weight=a["post_weight"], post_bias=a["post_bias"],
                                gate=a.get("gate"), pre_weight=a["pre_weight"], **kw)
    assert set(g) == set(a)
    _differences(loss, a, g, tol=2e-7)


def _naive_logprobs(z):
    m = max(z)
    s = sum(math.exp(v - m) for v in z)
    lp = [(v - m) - math.log(s) for v in z]
    return m + math.log(s), lp, -sum(math.exp(v) * v for v in lp if v > -math.inf)


def test_logprobs():
    r = _rng(3)
    z = np.round(r.standard_normal((5, 7)) * 3)  # ties
    z[1, [0, 4]] = -np.inf
    z[2, 1:] = -np.inf
    z[3] = -3.0e38
    targets = np.array([2, 4, 0, 6, -1])
    out = oracle.logprobs(z, targets, scale=0.8, top=7)
    for i in range(5):
        lse, lp, ent = _naive_logprobs([0.8 * v for v in z[i]])
        assert abs(out["lse"][i] - lse) <= 1e-12 * abs(lse) + 1e-12 and abs(out["entropy"][i] - ent) < 1e-12
        want = 0.0 if targets[i] < 0 else lp[targets[i]]
        assert out["logprob"][i] == want or abs(out["logprob"][i] - want) < 1e-12
        ids = sorted(range(7), key=lambda j: (-z[i, j], j))
        assert out["top_ids"][i].tolist() == ids
        assert np.allclose(out["top_logprobs"][i], [lp[j] for j in ids], atol=1e-12)
    for row, lse in (([-np.inf] * 3, -np.inf), ([0.0, np.nan, 1.0], np.nan), ([0.0, np.inf, 1.0], np.nan)):
        o = oracle.logprobs(np.array([row]), [1], top=2)
        assert np.array_equal(o["lse"], [lse], equal_nan=True)
        assert np.array_equal(o["logprob"], [lse], equal_nan=True)
        assert o["top_ids"][0].tolist() == ([0, 1] if lse == -np.inf else [1, 2])
    assert oracle.logprobs(np.full((1, 3), -np.inf))["entropy"][0] == 0.0


def test_logprobs_gradient():
    r = _rng(4)
    z = r.standard_normal((3, 6)) * 2
    targets, scale = np.array([5, -1, 0]), 0.8
    g = {k: r.standard_normal(3) for k in ("logprob", "lse", "entropy")}

    def loss(z):
        o = oracle.logprobs(z, targets, scale=scale)
        return float(sum((g[k] * o[k]).sum() for k in g))

    d = oracle.logprobs_grad(z, targets, dlogprob=g["logprob"], dlse=g["lse"], dentropy=g["entropy"], scale=scale)
    _differences(loss, dict(z=z), dict(z=d))
    z[0, [1, 3]] = -np.inf  # what is masked has no gradient, and the others' are those without it
    d = oracle.logprobs_grad(z, targets, dlogprob=g["logprob"], dentropy=g["entropy"], scale=scale)
    keep = [0, 2, 4, 5]
    few = oracle.logprobs_grad(z[:1, keep], [3], dlogprob=g["logprob"][:1], dentropy=g["entropy"][:1], scale=scale)
    assert not d[0, [1, 3]].any() and np.abs(d[0, keep] - few[0]).max() < 1e-15
    assert not oracle.logprobs_grad(np.full((1, 4), -np.inf), [2], dlogprob=[1.0], dentropy=[1.0]).any()


def test_mistakes_show():
    """What the checks above would catch: a gate of the neighbouring sample, the scale left out of the gradient."""
    r = _rng(5)
    h, x, gate = r.standard_normal((4, 3)), r.standard_normal((4, 3)), r.standard_normal((2, 3))
    assert not np.allclose(oracle.block_norms(h, x, gate=gate)[0], oracle.block_norms(h, x, gate=gate[::-1])[0])
    z = r.standard_normal((2, 5))
    d = oracle.logprobs_grad(z, [0, 1], dlogprob=[1.0, 1.0], scale=0.5)
    assert not np.allclose(d, oracle.logprobs_grad(z * 0.5, [0, 1], dlogprob=[1.0, 1.0]))
