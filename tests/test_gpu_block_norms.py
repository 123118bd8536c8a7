"""GPU parity of the norms around a block (forward and gradient) against the
fp64 oracle.

Tolerance, element by element.  u = 2^-24 is half a step of fp32; a sum of n
terms by threads of 8 to 32 terms, shuffles and up to 64 partial sums loses at
most (32 + 5 + 64) u of the sum of the terms' sizes, taken here as K = 128 u.  A
norm's mean is off by K mean|t|, its mean square by 2 K of it, so the root by K:
a normalised value t^ is off by K (|t^| + mean|t| r) with a few roundings of its
own, for which K has room.  Through weight and bias that is K (|w| (|t^| + m r) +
|b|), m = mean|t|.  The second norm's input carries the first one's error e; its
output moves by at most r |w| (e + mean e + |t^| rms e).  The gradient's terms are
bounded by the same rule (every factor's size times K, the sums' terms in size),
the column sums over T rows by (T + 128) u of the sum of sizes and K of each
term.  Last, half a step of the output's type."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf, inputs
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 1e-44}
U = 2.0 ** -24
K = 128 * U
EPS = 1e-5


def _round(a, dt):
    a = np.asarray(a, dtype=np.float32)
    return {"bf16": inputs.round_to_bf16, "fp16": lambda v: v.astype(np.float16).astype(np.float32),
            "fp32": lambda v: v}[dt](a)


def _dev(a, dt="fp32"):
    torch = torch_cuda()
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dt])


def _host(t):
    return t.double().cpu().numpy()


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _check(got, ref, slack, dt, what):
    bound = HALF[dt] * (np.abs(ref) + slack) + slack + TINY[dt]
    err = np.abs(_host(got) - ref)
    assert err.shape == bound.shape and np.all(np.isfinite(err)), f"{what}: shape or non-finite"
    worst = np.argmax(err - bound)
    assert err.flat[worst] <= bound.flat[worst], (
        f"{what}: {err.flat[worst]:.3e} > {bound.flat[worst]:.3e} at {np.unravel_index(worst, err.shape)}, "
        f"ref {ref.flat[worst]:.4f}")


def _size(v, shape=1.0):
    return shape if v is None else np.abs(np.asarray(v, np.float64))


def _normed(kind, t, weight, bias, e):
    """Bound of the error of a norm's output, for an input t off by e."""
    t = np.asarray(t, np.float64)
    if kind == "none":
        return e * _size(weight)
    hat, r = oracle.norm_rows(kind, t, EPS)
    m = np.abs(t).mean(1, keepdims=True)
    rms = np.sqrt((e * e).mean(1, keepdims=True)) if np.ndim(e) else e
    mean = e.mean(1, keepdims=True) if np.ndim(e) else e
    return _size(weight) * (K * (np.abs(hat) + m * r) + r * e + r * mean + np.abs(hat) * r * rms) + \
        2 * U * _size(bias, 0.0)


def _hat_error(kind, t):
    if kind == "none":
        return 0.0
    hat, r = oracle.norm_rows(kind, t, EPS)
    return K * (np.abs(hat) + np.abs(np.asarray(t, np.float64)).mean(1, keepdims=True) * r)


# rows, columns: one token, a few, short rows, rows of a warp, odd, wide, wider than one CTA of the gradient
SHAPES = [(1, 4096), (3, 8), (7, 64), (1000, 64), (33, 96), (500, 128), (21, 248), (300, 1000), (64, 1111), (5, 3),
          (2, 1), (9, 2056), (40, 4096), (6, 5000), (12, 8192), (3, 9999), (2, 16384), (2, 32768), (1, 32765)]
NORMS = [("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("rms", "none"), ("layer", "rms"), ("none", "none")]


def _case(shape, dt, post, pre, gates, shift, seed=0):
    T, N = shape
    r = _rng(seed + T + N)
    c = dict(h=_round(r.standard_normal(shape) * 0.7 + 0.3, dt), x=_round(r.standard_normal(shape) * 1.5 - 0.2, dt))
    v = {}
    for name, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            v[name + "_weight"] = (1 + 0.3 * r.standard_normal(N)).astype(np.float32)
            if shift:
                v[name + "_bias"] = (0.3 * r.standard_normal(N)).astype(np.float32)
    gate = _round(r.standard_normal((gates, N)) * 0.5 + 0.5, dt) if gates else None
    return c, v, gate, dict(post=post, pre=pre, scale=0.75, alpha=1.25, eps=EPS)


def _gates(T):
    """None, one for all, one for each, and a divisor between."""
    some = [d for d in range(2, T) if T % d == 0]
    return sorted({0, 1, T} | set(some[len(some) // 2:len(some) // 2 + 1]))


def _forward_bounds(c, v, gate, kw):
    w = kw["scale"] * (np.abs(oracle.block_norms(c["h"], None, gate=gate, **{k: a for k, a in v.items() if "post" in k},
                                                 post=kw["post"], scale=1.0)[0]))
    g = 1.0 if gate is None else np.repeat(np.abs(gate.astype(np.float64)), len(c["h"]) // len(gate), 0)
    x = kw["alpha"] * np.abs(c["x"].astype(np.float64)) if c["x"] is not None else 0.0
    e = kw["scale"] * g * _normed(kw["post"], c["h"], v.get("post_weight"), v.get("post_bias"), 0.0) + 4 * U * (w + x)
    return e


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("norms", NORMS, ids="-".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, norms, dt):
    torch = torch_cuda()
    for gates, shift in ((g, s) for g in _gates(shape[0]) for s in (False, True)):
        c, v, gate, kw = _case(shape, dt, *norms, gates, shift)
        dv = {k: _dev(a) for k, a in v.items()}
        h, x = _dev(c["h"], dt), _dev(c["x"], dt)
        xo, y = cf.stitch_block_norms(h, x, gate=_dev(gate, dt), **dv, **kw)
        ref_x, ref_y = oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)
        e = _forward_bounds(c, v, gate, kw)
        _check(xo, ref_x, e, dt, "x_out")
        if norms[1] == "none":
            assert y is None
        else:
            _check(y, ref_y, _normed(norms[1], ref_x, v.get("pre_weight"), v.get("pre_bias"), e) +
                   2 * U * np.abs(ref_y), dt, "y")
            # in place, either way round, and without a stream
            x2, h2 = x.clone(), h.clone()
            cf.stitch_block_norms(h2, x2, gate=_dev(gate, dt), **dv, **kw, out=x2, norm_out=h2)
            assert torch.equal(x2, xo) and torch.equal(h2, y)
            xo, y = cf.stitch_block_norms(h, None, gate=_dev(gate, dt), **dv, **kw)
            ref_x, ref_y = oracle.block_norms(c["h"], None, gate=gate, **v, **kw)
            e = _forward_bounds(dict(c, x=None), v, gate, kw)
            _check(xo, ref_x, e, dt, "x_out without a stream")


def _grad_bounds(dy, dxo, c, xo, v, gate, kw):
    """Bounds of the gradient's errors, by the rule above; the keys of the oracle's gradient."""
    h, xo = np.asarray(c["h"], np.float64), np.asarray(xo, np.float64)
    T, N = h.shape
    d, e = (np.zeros_like(h), np.zeros_like(h)) if dxo is None else (np.asarray(dxo, np.float64), np.zeros_like(h))
    out = {}

    def through(kind, t, g, eg):
        """Size and error of a norm's input gradient for one behind it, g, off by eg."""
        if kind == "none":
            return np.abs(g) + 0 * t, eg + 2 * U * np.abs(g)
        hat, r = oracle.norm_rows(kind, t, EPS)
        eh = _hat_error(kind, t)
        ga, ha = np.abs(g), np.abs(hat)
        mg = ga.mean(1, keepdims=True) if kind == "layer" else 0.0
        mgh = (ga * ha).mean(1, keepdims=True)
        size = r * (ga + mg + ha * mgh)
        em = (eg.mean(1, keepdims=True) + K * mg) if kind == "layer" else 0.0
        emh = (eg * ha + ga * eh).mean(1, keepdims=True) + K * mgh
        return size, r * (eg + em + ha * emh + eh * mgh) + K * size

    if dy is not None:
        dy = np.asarray(dy, np.float64)
        hat, _ = oracle.norm_rows(kw["pre"], xo, EPS)
        eh = _hat_error(kw["pre"], xo)
        rows = (T + 128) * U
        out["pre_weight"] = (np.abs(dy) * eh).sum(0) + rows * (np.abs(dy * hat)).sum(0)
        out["pre_bias"] = rows * np.abs(dy).sum(0)
        g = dy * (1.0 if v.get("pre_weight") is None else v["pre_weight"].astype(np.float64))
        size, e2 = through(kw["pre"], xo, g, U * np.abs(g))
        e = e2 + 2 * U * (np.abs(d) + size)
        hat2, r = oracle.norm_rows(kw["pre"], xo, EPS)
        d = oracle.block_norms_grad(dy, dxo, h, xo, post="none", pre=kw["pre"], pre_weight=v.get("pre_weight"),
                                    eps=EPS)["x"]
    out["x"] = kw["alpha"] * e + 2 * U * np.abs(kw["alpha"] * d)
    hat, _ = oracle.norm_rows(kw["post"], h, EPS)
    eh = _hat_error(kw["post"], h)
    ga = 1.0 if gate is None else np.repeat(np.abs(gate.astype(np.float64)), T // len(gate), 0)
    s = kw["scale"]
    dpa, edp = s * ga * np.abs(d), s * ga * e + 4 * U * s * ga * np.abs(d)
    rows = (T + 128) * U
    out["post_weight"] = (edp * np.abs(hat) + dpa * eh).sum(0) + rows * (dpa * np.abs(hat)).sum(0)
    out["post_bias"] = edp.sum(0) + rows * dpa.sum(0)
    w, b = _size(v.get("post_weight")), _size(v.get("post_bias"), 0.0)
    if gate is not None:
        terms = s * ((e + 4 * U * np.abs(d)) * (np.abs(hat) * w + b) + np.abs(d) * eh * w) + \
            rows * s * np.abs(d) * (np.abs(hat) * w + b)
        out["gate"] = terms.reshape(len(gate), -1, N).sum(1)
    out["h"] = through(kw["post"], h, dpa * w, edp * w + U * dpa * w)[1]
    return out


KEYS = ("h", "x", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("norms", NORMS, ids="-".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(shape, norms, dt):
    torch = torch_cuda()
    T, N = shape
    ws = cf.new_workspace(cf.cf_stitch_block_norms_grad_workspace_size(T, N))
    for gates, shift in ((g, s) for g in _gates(T) for s in (False, True)):
        c, v, gate, kw = _case(shape, dt, *norms, gates, shift)
        r = _rng(5)
        dy = None if norms[1] == "none" else _round(r.standard_normal(shape), dt)
        dxo = _round(r.standard_normal(shape), dt) if dy is None or gates != 1 else None
        xo = _round(oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], dt)
        args = (_dev(dy, dt), _dev(dxo, dt), _dev(c["h"], dt), _dev(xo, dt))
        dv = {k: _dev(a) for k, a in v.items()}
        got = cf.stitch_block_norms_grad(*args, gate=_dev(gate, dt), **dv, **kw, workspace=ws)
        okw = {k: a for k, a in v.items() if k != "pre_bias"}
        ref = oracle.block_norms_grad(dy, dxo, c["h"], xo, gate=gate, **okw, **kw)
        bounds = _grad_bounds(dy, dxo, c, xo, v, gate, kw)
        for k, t in zip(KEYS, got):
            wanted = k in ("h", "x") or k in v or (k == "gate" and gate is not None)
            assert (t is not None) == wanted, k
            if wanted:
                _check(t, ref[k], bounds[k], dt if k in ("h", "x", "gate") else "fp32", f"d{k} {gates} {shift}")
        again = cf.stitch_block_norms_grad(*[None if a is None else a.clone() for a in args], gate=_dev(gate, dt), **dv,
                                           **kw, workspace=ws)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
        # in place of what came in; the stream's gradient not wanted
        out = [args[2], args[1] if args[1] is not None else args[0]] + [None] * 5
        same = cf.stitch_block_norms_grad(*args, gate=_dev(gate, dt), **dv, **kw, workspace=ws, out=out)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, same))


# more rows than CTAs, of more than 8192 columns: several rows of a ring for each of them
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("norms", [("rms", "rms"), ("layer", "layer")], ids="-".join)
@pytest.mark.parametrize("shape", [(400, 8200), (330, 10001), (310, 16384)], ids=str)
def test_wide_rows(shape, norms, dt):
    ws = cf.new_workspace(cf.cf_stitch_block_norms_grad_workspace_size(*shape))
    for gates, shift in ((0, False), (shape[0], True), (shape[0] // 10, False), (1, True)):
        c, v, gate, kw = _case(shape, dt, *norms, gates, shift)
        dv, g = {k: _dev(a) for k, a in v.items()}, _dev(gate, dt)
        xo, y = cf.stitch_block_norms(_dev(c["h"], dt), _dev(c["x"], dt), gate=g, **dv, **kw)
        ref_x, ref_y = oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)
        e = _forward_bounds(c, v, gate, kw)
        _check(xo, ref_x, e, dt, "x_out")
        _check(y, ref_y, _normed(norms[1], ref_x, v.get("pre_weight"), v.get("pre_bias"), e) + 2 * U * np.abs(ref_y), dt,
               "y")
        x16 = _round(ref_x, dt)
        dy = _round(_rng(5).standard_normal(shape), dt)
        got = cf.stitch_block_norms_grad(_dev(dy, dt), None, _dev(c["h"], dt), _dev(x16, dt), gate=g, **dv, **kw,
                                         workspace=ws)
        okw = {k: a for k, a in v.items() if k != "pre_bias"}
        ref = oracle.block_norms_grad(dy, None, c["h"], x16, gate=gate, **okw, **kw)
        bounds = _grad_bounds(dy, None, c, x16, v, gate, kw)
        for k, t in zip(KEYS, got):
            if t is not None:
                _check(t, ref[k], bounds[k], dt if k in ("h", "x", "gate") else "fp32", f"d{k} {gates} {shift}")


# A LayerNorm whose mean is far from zero, whose parts have means of their own, and whose first part lies far from the
# others: squares about the mean of a part, put together, lose nothing of the small ones.
@pytest.mark.parametrize("N", [64, 300, 2056, 4096, 8192, 9999, 16384, 32768])
def test_means_of_parts(N):
    r = _rng(N)
    h = r.standard_normal((12, N))
    h[0] += 1000.0
    h[1] += 100.0 * (np.arange(N) // 256)
    h[2, :min(512, N // 2)] += 3000.0
    h[3, -min(512, N // 2):] -= 3000.0
    h[4] = 5.0 + 1e-3 * h[4]
    h[5, 0] = 1e4
    h[6, -1] = 1e4
    h[7] *= 1e-4
    h = h.astype(np.float32)
    x = np.zeros_like(h)
    w, b = r.standard_normal((2, N)).astype(np.float32)
    xo, y = cf.stitch_block_norms(_dev(h), _dev(x), post_weight=_dev(w), post_bias=_dev(b), pre_weight=_dev(w),
                                  pre_bias=_dev(b), post="layer", pre="layer", eps=EPS)
    ref_x, ref_y = oracle.block_norms(h, x, post_weight=w, post_bias=b, pre_weight=w, pre_bias=b, post="layer",
                                      pre="layer", eps=EPS)
    e = _normed("layer", h, w, b, 0.0) + 4 * U * np.abs(ref_x)
    _check(xo, ref_x, e, "fp32", "x_out")
    _check(y, ref_y, _normed("layer", ref_x, w, b, e) + 2 * U * np.abs(ref_y), "fp32", "y")


def test_nans_stay_in_their_rows():
    torch = torch_cuda()
    c, v, gate, kw = _case((40, 200), "bf16", "layer", "rms", 8, True)
    h, x = _dev(c["h"], "bf16"), _dev(c["x"], "bf16")
    dv = {k: _dev(a) for k, a in v.items()}
    g = _dev(gate, "bf16")
    clean = cf.stitch_block_norms(h, x, gate=g, **dv, **kw)
    dclean = cf.stitch_block_norms_grad(h, x, h, clean[0], gate=g, **dv, **kw)
    h[7, 3], x[20, 199] = float("nan"), float("inf")
    rest = [i for i in range(40) if i not in (7, 20)]
    out = cf.stitch_block_norms(h, x, gate=g, **dv, **kw)
    for a, b in zip(out, clean):
        assert torch.equal(a[rest], b[rest]) and a[7].isnan().all()
    d = cf.stitch_block_norms_grad(h, x, h, out[0], gate=g, **dv, **kw)
    for a, b in zip(d[:2], dclean[:2]):
        assert torch.equal(a[rest], b[rest]) and a[7].isnan().all()
    assert torch.equal(d[2][[0, 2, 3, 5, 6, 7]], dclean[2][[0, 2, 3, 5, 6, 7]])  # the other samples' gates


def test_equal_values_and_large_ones():
    """A constant row (a variance of zero), and rows whose mean is far larger than what is around it."""
    T, N = 3, 512
    h = np.full((T, N), 3.0, np.float32)
    h[1] = 1000.0 + np.arange(N) % 7
    h[2] = 1e-3
    for post in ("layer", "rms"):
        kw = dict(post=post, pre="layer", scale=1.0, alpha=0.0, eps=EPS)
        xo, y = cf.stitch_block_norms(_dev(h), None, **kw)
        ref_x, ref_y = oracle.block_norms(h, None, **kw)
        e = _normed(post, h, None, None, 0.0) + 4 * U * np.abs(ref_x)
        _check(xo, ref_x, e, "fp32", post)
        _check(y, ref_y, _normed("layer", ref_x, None, None, e) + 2 * U * np.abs(ref_y), "fp32", post)


def test_no_rows_and_no_columns():
    torch = torch_cuda()
    e = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    xo, y = cf.stitch_block_norms(e, e, post="rms", pre="rms", pre_weight=w)
    assert xo.shape == y.shape == (0, 64)
    d = cf.stitch_block_norms_grad(e, e, e, e, post="rms", post_weight=w, pre="rms", pre_weight=w)
    assert not d[3].any() and not d[5].any() and d[3].shape == (64,)
    n = torch.zeros(3, 0, device="cuda")
    assert cf.stitch_block_norms(n, n, pre="rms")[1].shape == (3, 0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 1024, 9000])
@pytest.mark.parametrize("shift", [1, 3, 7])
def test_gradient_of_unaligned_rows(N, dt, shift):
    """Tensors that start anywhere in memory, each elsewhere."""
    torch = torch_cuda()
    c, v, gate, kw = _case((30, N), dt, "rms", "rms", 3, False)
    dv = {k: _dev(a) for k, a in v.items()}

    def odd(a, by):
        t = _dev(a, dt)
        out = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[by % 8:by % 8 + t.numel()].view(t.shape)
        return out.copy_(t)

    r = _rng(3)
    dy, dxo = _round(r.standard_normal((30, N)), dt), _round(r.standard_normal((30, N)), dt)
    xo = _round(oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], dt)
    args = [odd(a, shift * (i + 1)) for i, a in enumerate((dy, dxo, c["h"], xo))]
    got = cf.stitch_block_norms_grad(*args, gate=odd(gate, 5), **dv, **kw)
    ref = oracle.block_norms_grad(dy, dxo, c["h"], xo, gate=gate, **v, **kw)
    bounds = _grad_bounds(dy, dxo, c, xo, v, gate, kw)
    for k, t in zip(KEYS, got):
        if t is not None:
            _check(t, ref[k], bounds[k], dt if k in ("h", "x", "gate") else "fp32", k)
    out, y = cf.stitch_block_norms(args[2], odd(c["x"], 2), gate=odd(gate, 5), **dv, **kw)
    ref_x, ref_y = oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)
    e = _forward_bounds(c, v, gate, kw)
    _check(out, ref_x, e, dt, "x_out")
    _check(y, ref_y, _normed("rms", ref_x, v["pre_weight"], None, e) + 2 * U * np.abs(ref_y), dt, "y")


def test_unaligned_rows():
    """Tensors that start anywhere in memory."""
    torch = torch_cuda()
    c, v, gate, kw = _case((6, 64), "bf16", "rms", "layer", 2, True)
    dv = {k: _dev(a) for k, a in v.items()}
    h, x, g = _dev(c["h"], "bf16"), _dev(c["x"], "bf16"), _dev(gate, "bf16")
    want = cf.stitch_block_norms(h, x, gate=g, **dv, **kw)
    odd = torch.empty(6 * 64 + 1, dtype=h.dtype, device="cuda")[1:].view(6, 64)
    odd.copy_(h)
    ref_x, ref_y = oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)
    e = _forward_bounds(c, v, gate, kw)
    got = cf.stitch_block_norms(odd, x, gate=g, **dv, **kw)
    for pair in (want, got):
        _check(pair[0], ref_x, e, "bf16", "x_out")
        _check(pair[1], ref_y, _normed("layer", ref_x, v["pre_weight"], v["pre_bias"], e), "bf16", "y")


def test_wrapper_refusals():
    torch = torch_cuda()
    h, w = torch.zeros(4, 64, device="cuda"), torch.zeros(64, device="cuda")
    for f, match in ((lambda: cf.stitch_block_norms(h, h[:2]), "x has shape"),
                     (lambda: cf.stitch_block_norms(h, h, post="batch"), "post"),
                     (lambda: cf.stitch_block_norms(h, h, post_weight=w), "post is no norm"),
                     (lambda: cf.stitch_block_norms(h, h, gate=h[:3]), "divide"),
                     (lambda: cf.stitch_block_norms(h, h, gate=h[:2].half()), "gate has dtype"),
                     (lambda: cf.stitch_block_norms(h, h, norm_out=h), "norm_out"),
                     (lambda: cf.stitch_block_norms(h.t(), None), "contiguous"),
                     (lambda: cf.stitch_block_norms(h.double(), None), "dtype"),
                     (lambda: cf.stitch_block_norms(h, h, pre="rms", pre_weight=w[:3]), "pre_weight"),
                     (lambda: cf.stitch_block_norms_grad(None, h, h, h, pre="rms"), "dy"),
                     (lambda: cf.stitch_block_norms_grad(h, h, h, h), "dy"),
                     (lambda: cf.stitch_block_norms_grad(h, h[:1], h, h, pre="rms"), "dx_out")):
        with pytest.raises(ValueError, match=match):
            f()
    with pytest.raises(cf.CfError):
        cf.stitch_block_norms(h, h, pre="rms", out=h, norm_out=h)
