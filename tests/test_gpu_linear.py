"""GPU parity of the dense layer (forward and gradients) against the fp64
oracle, through the C ABI and the torch-level calls.

Tolerance, element by element: half a step of the 16-bit output (at least half
its smallest subnormal), plus the fp32 accumulation.  A sum of n products in any
order is off by at most n 2^-23 sum|a b|; the bias and the residual add one
rounding each, 2^-24 of a value no larger than sum|a b| + |bias| + |residual|.
The activations' slopes are at most 1.13 and carry the product's error; the
functions' own errors (ex2.approx of an argument rounded to fp32, a quotient
within 2 steps) stay below 2^-16 of the value where the exponent's argument is
below 64 in size, and beyond that the value is z or below 1e-10.

The gradients start from dZ = dY act'(Z), which the products see rounded to 16
bits: half a step of each dZ, and 2^-16 |dY| (1 + |Z|) for the slope (of
p + z p (1 - p) u' each term loses that much of |z| p at the most)."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf, inputs
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25}
ACC = 2.0 ** -23
ACTS = ["none", "gelu_tanh", "silu", "relu"]


def _round(a, dt):
    a = np.asarray(a, dtype=np.float32)
    return inputs.round_to_bf16(a) if dt == "bf16" else a.astype(np.float16).astype(np.float32)


def _dev(a, dt="fp32"):
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dt])


def _host(t):
    return t.double().cpu().numpy()


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _check(got, ref, slack, half, tiny, what):
    bound = half * np.abs(ref) + slack + tiny
    err = np.abs(got - ref)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), f"{what}: shape or non-finite"
    if err.size:
        worst = np.argmax(err - bound)
        assert err.flat[worst] <= bound.flat[worst], (
            f"{what}: {err.flat[worst]:.3e} > {bound.flat[worst]:.3e} at {np.unravel_index(worst, err.shape)}, "
            f"ref {ref.flat[worst]:.4f}")


def _status(ws):
    st, info = cf.cf_get_device_status(ws)
    assert st == cf.CF_OK, (cf.status_string(st), hex(info))


# M, K, N: one token, a few, ragged, more than a row tile, more than a wave of tiles
SHAPES = [(1, 64, 128), (1, 1024, 2048), (3, 8, 8), (17, 136, 200), (129, 72, 136), (257, 320, 520), (1003, 1000, 264),
          (700, 64, 5344), (2048, 512, 1024)]
TUNINGS = {"auto": {}, "n16": dict(n_slice=16), "n64": dict(n_slice=64, cluster_m=1, stages=2),
           "n256": dict(n_slice=256, cluster_m=1, max_clusters=3),
           "pair128": dict(n_slice=128, cluster_m=2, max_clusters=2), "pair256": dict(n_slice=256, cluster_m=2)}


def _case(shape, dt, seed=0):
    M, K, N = shape
    r = _rng(seed + M + K + N)
    X = _round(r.standard_normal((M, K)), dt)
    W = _round(r.standard_normal((K, N)) * K ** -0.5, dt)
    return X, W, r.standard_normal(N).astype(np.float32), _round(r.standard_normal((M, N)), dt)


def _forward(X, W, b, R, act, dt, tun=None, **kw):
    M, K, N = *X.shape, W.shape[1]
    ws = cf.new_workspace(cf.cf_gemm_linear_workspace_size(M, N, K))
    y = cf.gemm_linear(_dev(X, dt), _dev(W, dt), None if b is None else _dev(b), act=act,
                       residual=None if R is None else _dev(R, dt), workspace=ws, tuning=tun, **kw)
    _status(ws)
    return y


def _check_forward(y, z, X, W, b, R, act, dt):
    Y, Z = oracle.gemm_linear(X, W, b, act=act, residual=R)
    b0, r0 = (0.0 if v is None else np.abs(np.asarray(v, np.float64)) for v in (b, R))
    zs = X.shape[1] * ACC * oracle.gemm_linear(np.abs(X), np.abs(W))[0] + 2.0 ** -24 * (np.abs(Z) + b0)
    if z is not None:
        _check(_host(z), Z, zs, HALF[dt], TINY[dt], "Z")
    own = oracle.activation(act, Z)
    ys = zs if act == "none" else 1.13 * zs + 2.0 ** -16 * np.abs(own) + 1e-10
    _check(_host(y), Y, ys + 2.0 ** -23 * (np.abs(own) + r0), HALF[dt], TINY[dt], "Y")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ACTS)
def test_forward(shape, dt, act):
    torch = torch_cuda()
    X, W, b, R = _case(shape, dt)
    z = torch.empty(R.shape, dtype=_dev(X[:1], dt).dtype, device="cuda")
    y = _forward(X, W, b, R, act, dt, preact=z)
    _check_forward(y, z, X, W, b, R, act, dt)
    assert torch.equal(y, _forward(X, W, b, R, act, dt))  # without the pre-activation: the same bits
    for bb, rr in ((None, None), (b, None), (None, R)):
        _check_forward(_forward(X, W, bb, rr, act, dt), None, X, W, bb, rr, act, dt)


@pytest.mark.parametrize("tun", [t for t in TUNINGS if t != "auto"])
@pytest.mark.parametrize("shape", SHAPES[2:], ids=str)
def test_forward_tiles(shape, tun):
    X, W, b, R = _case(shape, "bf16")
    _check_forward(_forward(X, W, b, R, "silu", "bf16", cf.tuning(**TUNINGS[tun])), None, X, W, b, R, "silu", "bf16")


def test_residual_in_place():
    torch = torch_cuda()
    for shape in SHAPES:
        X, W, b, R = _case(shape, "fp16")
        want = _forward(X, W, b, R, "gelu_tanh", "fp16")
        r = _dev(R, "fp16")
        got = cf.gemm_linear(_dev(X, "fp16"), _dev(W, "fp16"), _dev(b), act="gelu_tanh", residual=r, out=r)
        assert got is r and torch.equal(got, want)


def test_infinities_stay_in_their_rows():
    X, W, b, R = _case((40, 64, 72), "bf16")
    clean = _host(_forward(X, W, b, R, "silu", "bf16"))
    X[3, 5], X[39, 0], R[7, 9] = np.inf, np.nan, -np.inf
    y = _host(_forward(X, W, b, R, "silu", "bf16"))
    rest = np.setdiff1d(np.arange(40), [3, 39])
    assert y[7, 9] == -np.inf and np.isnan(y[39]).all() and not np.isfinite(y[3]).all()
    y[7, 9] = clean[7, 9]
    assert np.array_equal(y[rest], clean[rest])


@pytest.mark.parametrize("act", ACTS)
def test_ends_of_the_activation(act):
    """Pre-activations of every size, by a product with the identity."""
    v = np.array([0.0, -0.0, 1e-3, -1e-3, 3.0, -3.0, -7.5, 12.0, -12.0, 80.0, -80.0, 100.0, -100.0, 3e4, -3e4, 6e4],
                 dtype=np.float32)
    X, W = np.zeros((16, 16), np.float32), np.eye(16, dtype=np.float32)
    X[:] = _round(v, "fp16")  # (what the kernel sees)
    y = _forward(X, W, None, None, act, "fp16")
    _check_forward(y, None, X, W, None, None, act, "fp16")
    dz = _dev(np.zeros((16, 16)), "fp16")
    cf.gemm_linear_grad(_dev(np.ones((16, 16)), "fp16"), _dev(X, "fp16"), _dev(W, "fp16"), act=act,
                        preact=_dev(X, "fp16"), dz=dz) if act != "none" else dz.fill_(1)
    z = _round(X, "fp16")
    _check(_host(dz), oracle.activation_slope(act, z), 2.0 ** -16 * (1 + np.minimum(np.abs(z), 16)), HALF["fp16"],
           TINY["fp16"], "slope")


def _grad_case(shape, dt):
    X, W, _, _ = _case(shape, dt)
    r = _rng(7)
    M, K, N = shape
    return X, W, _round(r.standard_normal((M, N)) * 1.5, dt), _round(r.standard_normal((M, N)), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ACTS)
def test_gradient(shape, dt, act):
    torch = torch_cuda()
    X, W, Z, dY = _grad_case(shape, dt)
    M, K, N = shape
    ws = cf.new_workspace(cf.cf_gemm_linear_workspace_size(M, N, K))
    z = None if act == "none" else _dev(Z, dt)
    args = (_dev(dY, dt), _dev(X, dt), _dev(W, dt))
    got = cf.gemm_linear_grad(*args, act=act, preact=z, workspace=ws)
    _status(ws)
    dX, dW, db = oracle.gemm_linear_grad(dY, X, W, act=act, preact=Z)
    dZ = dY if act == "none" else dY * oracle.activation_slope(act, Z)
    own = np.zeros_like(dZ) if act == "none" else 2.0 ** -16 * np.abs(dY) * (1 + np.abs(Z))  # of dZ before rounding
    off = own if act == "none" else own + HALF[dt] * (np.abs(dZ) + own) + TINY[dt]
    full = np.abs(dZ) + off
    _check(_host(got[0]), dX, off @ np.abs(W).T + N * ACC * (full @ np.abs(W).T), HALF[dt], TINY[dt], "dX")
    _check(_host(got[1]), dW, np.abs(X).T @ off + M * ACC * (np.abs(X).T @ full), HALF[dt], TINY[dt], "dW")
    _check(_host(got[2]), db, own.sum(0) + M * ACC * full.sum(0), 2.0 ** -24, 0.0, "dbias")
    again = cf.gemm_linear_grad(*args, act=act, preact=z, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # equal calls give equal bits
    # each alone, and dZ in the place of Z
    for i, name in enumerate(("input", "weight", "bias")):
        one = dict(input=False, weight=False, bias=False)
        one[name] = True
        zz = None if z is None else z.clone()
        part = cf.gemm_linear_grad(args[0], args[1] if i == 1 else None, args[2] if i != 1 else None, act=act,
                                   preact=zz, dz=zz, workspace=ws, **one)
        assert torch.equal(part[i], got[i]) and sum(p is not None for p in part) == 1


# many rows: tiles of CTA pairs that are cut to fill the last round
@pytest.mark.parametrize("shape", [(8191, 128, 2048), (5003, 520, 2056), (8191, 2048, 128)], ids=str)
def test_many_rows(shape):
    X, W, b, R = _case(shape, "bf16")
    torch = torch_cuda()
    z = torch.empty(R.shape, dtype=torch.bfloat16, device="cuda")
    y = _forward(X, W, b, R, "silu", "bf16", preact=z)
    _check_forward(y, z, X, W, b, R, "silu", "bf16")
    X, W, Z, dY = _grad_case(shape, "bf16")
    M, K, N = shape
    dX, dW, db = cf.gemm_linear_grad(_dev(dY, "bf16"), _dev(X, "bf16"), _dev(W, "bf16"))
    rX, rW, rb = oracle.gemm_linear_grad(dY, X, W)
    size = np.abs(dY)
    _check(_host(dX), rX, N * ACC * (size @ np.abs(W).T), HALF["bf16"], TINY["bf16"], "dX")
    _check(_host(dW), rW, M * ACC * (np.abs(X).T @ size), HALF["bf16"], TINY["bf16"], "dW")
    _check(_host(db), rb, M * ACC * size.sum(0), 2.0 ** -24, 0.0, "dbias")


def test_no_rows():
    torch = torch_cuda()
    X, W = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 72, dtype=torch.bfloat16,
                                                                             device="cuda")
    assert cf.gemm_linear(X, W).shape == (0, 72)
    dX, dW, db = cf.gemm_linear_grad(torch.zeros(0, 72, dtype=torch.bfloat16, device="cuda"), X, W)
    assert dX.shape == (0, 64) and not dW.any() and not db.any() and dW.shape == (64, 72)


def test_wrapper_refusals():
    torch = torch_cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    X, W, Y = torch.zeros(4, 64, **bf), torch.zeros(64, 72, **bf), torch.zeros(4, 72, **bf)
    for f, match in ((lambda: cf.gemm_linear(X, W, act="tanh"), "activation"),
                     (lambda: cf.gemm_linear(X, W.t()), "W"),
                     (lambda: cf.gemm_linear(X, W, Y[0]), "bias"),
                     (lambda: cf.gemm_linear(X, W, residual=Y[:3]), "residual"),
                     (lambda: cf.gemm_linear(X.float(), W.float()), "X"),
                     (lambda: cf.gemm_linear_grad(Y, X, W, act="silu"), "preact"),
                     (lambda: cf.gemm_linear_grad(Y, X, W, preact=Y), "preact"),
                     (lambda: cf.gemm_linear_grad(Y, X, None), "W"),
                     (lambda: cf.gemm_linear_grad(Y, None, None), "X"),
                     (lambda: cf.gemm_linear_grad(Y, X, W, out=(None, W.t(), None)), r"out\[1\]")):
        with pytest.raises(ValueError, match=match):
            f()
