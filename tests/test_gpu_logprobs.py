"""GPU parity of the log probabilities of given tokens (forward and gradient)
against the fp64 oracle.

Tolerance, with u = 2^-24.  d = (z - m) log2 e is rounded three times (the
difference, the scale's factor, the product) and 2^d is off by 2^-22 of its value
(ex2.approx) and 3 u |d| ln 2; so sum 2^d is off by 2^-22 + 3 u (mean |z - m| under
p) of itself plus what adding loses, at most (a thread's terms + 64) u, here 600 u:
about 2^-14.5 at the most.  The log of the sum is off by as much, absolutely: A =
600 u + 2^-22 + 3 u D with D the spread max - mean of z under p.  lse adds the
rounding of m scale and of itself, 2 u |lse|; a log probability 3 u |z - m| and u of
itself; the entropy the error of the weighted mean, (A + 3 u) D + A.
The gradient's p = exp(z - lse) is off by p (2 u |z - lse| + 2^-22 + 3 u); its terms
follow, with a few roundings of each, and half a step of the output."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf, inputs
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25, "fp32": 2e-38}
U = 2.0 ** -24
# rows, vocabulary, padding between rows
SHAPES = [(1, 1, 0), (2, 5, 0), (3, 33, 2), (40, 257, 0), (7, 1000, 0), (400, 1001, 23), (5, 4096, 0), (2, 8192, 3),
          (1, 50257, 0), (16, 32003, 1), (90, 20000, 0), (700, 3001, 0), (1, 262147, 0), (160, 100000, 0)]


def _round(a, dt):
    a = np.asarray(a, dtype=np.float32)
    return {"bf16": inputs.round_to_bf16, "fp16": lambda v: v.astype(np.float16).astype(np.float32),
            "fp32": lambda v: v}[dt](a)


def _dev(a, dt="fp32", pad=0):
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    t = t.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dt])
    if pad:
        wide = torch.full((t.shape[0], t.shape[1] + pad), 3.0, dtype=t.dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :t.shape[1]]
    return t


def _i64(a):
    return torch_cuda().tensor(np.asarray(a), dtype=torch_cuda().int64, device="cuda")


def _host(t):
    return t.double().cpu().numpy()


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _status(ws, want=cf.CF_OK):
    st, info = cf.cf_get_device_status(ws)
    assert st == want, (cf.status_string(st), hex(info))


def _within(got, ref, bound, what):
    got = _host(got)
    assert got.shape == ref.shape, what
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - ref) <= bound)
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {got[at]} against {ref[at]} at {at}, bound {np.broadcast_to(bound, ref.shape)[at]}")


def _bounds(z, scale, ref):
    """D and A of each row."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = z.astype(np.float64) * scale
        m = s.max(1)
        p = np.exp(s - ref["lse"][:, None])
        spread = np.where(p > 0, p * (m[:, None] - s), 0.0).sum(1)
        spread = np.where(np.isfinite(spread), spread, 0.0)
        m = np.where(np.isfinite(m), m, 0.0)
    return m, spread, 600 * U + 2.0 ** -22 + 3 * U * spread


def _check(got, z, targets, scale, top, what=""):
    if z.size > 1 << 18:  # the oracle sorts: of many long rows it takes some
        pick = np.unique(np.linspace(0, len(z) - 1, 24).astype(int))
        got, z = [None if g is None else g[pick] for g in got], z[pick]
        targets = None if targets is None else targets[pick]
    ref = oracle.logprobs(z, targets, scale=scale, top=top)
    m, D, A = _bounds(z, scale, ref)
    lp, lse, h, tl, ti = got
    with np.errstate(invalid="ignore"):
        _within(lse, ref["lse"], A + 2 * U * (np.abs(ref["lse"]) + np.abs(m)), what + " lse")
        if h is not None:
            _within(h, ref["entropy"], (A + 3 * U) * D + A + 2 * U * ref["entropy"], what + " entropy")
        if targets is not None:
            _within(lp, ref["logprob"], A + 5 * U * (np.abs(ref["logprob"]) + np.log(z.shape[1])), what + " logprob")
        if top:
            assert np.array_equal(ti.cpu().numpy(), ref["top_ids"]), what + " ids"
            _within(tl, ref["top_logprobs"], A[:, None] + 5 * U * (np.abs(ref["top_logprobs"]) + np.log(z.shape[1])),
                    what + " top")


def _case(shape, dt, kind, seed=0):
    T, V, _ = shape
    r = _rng(seed + T + V)
    z = r.standard_normal((T, V)) * 2.5
    t = r.integers(0, V, T)
    if kind == "masked":
        z[r.random((T, V)) < 0.6] = -np.inf
        z[np.arange(T), t] = r.standard_normal(T)
        t[r.random(T) < 0.3] = -1
    elif kind == "coarse":  # many equal logits
        z = np.round(z)
    elif kind == "far":  # a maximum far from zero
        z = z + 1000.0
    return _round(z, dt), t


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["plain", "masked", "coarse", "far"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, kind, dt):
    torch = torch_cuda()
    z, t = _case(shape, dt, kind)
    zd, td = _dev(z, dt, shape[2]), _i64(t)
    ws = cf.new_workspace(cf.cf_stitch_workspace_size(*z.shape))
    for scale, top in ((1.0, min(20, shape[1])), (0.7, min(1, shape[1])), (1.3, 0), (1.0, min(32, shape[1]))):
        got = cf.stitch_logprobs(zd, td, scale=scale, top=top, workspace=ws)
        _status(ws)
        _check(got, z, t, np.float64(np.float32(scale)), top, f"{scale} {top}")
        again = cf.stitch_logprobs(zd, td, scale=scale, top=top, workspace=ws)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
        # the parts alone
        part = cf.stitch_logprobs(zd, None, scale=scale, top=top, entropy=False)
        assert part[0] is None and part[2] is None
        _check(part, z, None, np.float64(np.float32(scale)), top, "parts")


def _ends(dt, V):
    """Rows at the ends of what there is."""
    low = {"bf16": -3.3895313892515355e38, "fp16": -65504.0, "fp32": -3.4028234663852886e38}[dt]
    r = _rng(9)
    z = r.standard_normal((12, V)).astype(np.float32)
    z[0] = -np.inf
    z[1] = low  # a mask of the type's lowest value that leaves nothing
    z[2, :] = low
    z[2, V // 2] = -np.inf
    z[3, :] = -np.inf
    z[3, V - 1] = 2.0  # one token left
    z[4, V // 3] = np.nan
    z[5, V - 1] = np.inf
    z[6, :] = 0.0
    z[6, ::2] = -0.0  # the zeros are equal
    z[7, :] = 7.0
    z[8, 1:] = low
    z[9] = np.arange(V) / V * 8  # ascending
    z[10] = z[9][::-1]
    z[11, [0, V - 1]] = [np.nan, np.inf]
    return _round(z, dt), np.array([1, 2, V // 2, V - 1, 0, 0, 1, V - 1, 0, V - 1, 0, 2])


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [40, 1003, 9000, 140000])
def test_ends(V, dt):
    z, t = _ends(dt, V)
    for rows in (slice(0, 12), *(slice(i, i + 1) for i in range(12))):  # with and without CTAs that share a row
        got = cf.stitch_logprobs(_dev(z[rows], dt), _i64(t[rows]), top=20)
        _check(got, z[rows], t[rows], 1.0, 20, str(rows))


@pytest.mark.parametrize("top", [1, 20, 32])
def test_large_logits_in_few_threads(top):
    """Large logits at a distance that puts them all in the windows of a few threads, more than the candidates' list
    holds, in ascending and descending order."""
    V = 1 << 20
    z = np.full((2, V), -5.0, np.float32)
    at = (np.arange(V) // 8) % 256 < 24
    z[0, at] = np.arange(at.sum()) % 251
    z[1, at] = np.arange(at.sum())[::-1]
    z = np.repeat(z, 160, 0)  # one CTA a row
    for dt in ("fp32", "bf16"):
        zr = _round(z, dt)
        got = cf.stitch_logprobs(_dev(zr, dt), None, top=top)
        pick = [0, 160, 319]
        _check([None if g is None else g[pick] for g in got], zr[pick], None, 1.0, top, dt)


# enough rows to fill the SMs with few threads each
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["plain", "masked", "coarse"])
@pytest.mark.parametrize("shape", [(4200, 70, 0), (2500, 4001, 0), (1100, 9003, 5), (1000, 30000, 0)], ids=str)
def test_many_rows(shape, kind, dt):
    z, t = _case(shape, dt, kind)
    for top in (1, 6, 32):
        _check(cf.stitch_logprobs(_dev(z, dt, shape[2]), _i64(t), top=top), z, t, 1.0, top, f"{top}")


# The threads that hold the top tokens have several windows of them, or as many others as good lie behind them.
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("top", [1, 4, 5, 32])
def test_equal_logits_on_the_bound(top, dt):
    r = _rng(top)
    z = _round(r.standard_normal((6, 20011)), dt)
    z[0, r.permutation(20011)[:700]] = 9.0
    z[1, ::977] = 9.0
    z[1, 5::977] = 9.5
    z[2, 8000:8000 + 64] = 9.0
    z[3, r.permutation(20011)[:2500]] = 9.0
    z[4] = -5.0
    z[4, -1] = -4.0
    z[5] = -np.inf
    z[5, 19990:19990 + top] = -1.0
    t = r.integers(0, 20011, 6)
    _check(cf.stitch_logprobs(_dev(z, dt), _i64(t), top=top), z, t, 1.0, top)


def test_targets_out_of_range():
    z, _ = _case((4, 100, 0), "fp32", "plain")
    ws = cf.new_workspace(cf.cf_stitch_workspace_size(4, 100))
    for bad in (100, -2, 1 << 40):
        got = cf.stitch_logprobs(_dev(z), _i64([3, bad, -1, 99]), workspace=ws)
        _status(ws, cf.CF_ERR_DEVICE_BOUNDS)
        _check(got, z, np.array([3, -1, -1, 99]), 1.0, 0)
        d = cf.stitch_logprobs_grad(_dev(z), _i64([3, bad, -1, 99]), got[1], _dev(np.ones(4)), workspace=ws)
        _status(ws, cf.CF_ERR_DEVICE_BOUNDS)
        _within(d, oracle.logprobs_grad(z, [3, -1, -1, 99], dlogprob=np.ones(4)), 1e-6, "gradient")


def _grad_bound(z, t, scale, lse, ent, dlp, dl, dh, dt, ref):
    zero = np.zeros(len(z))
    dlp, dl, dh = (zero if v is None else np.abs(v.astype(np.float64)) for v in (dlp, dl, dh))
    dlp = np.where(t < 0, 0.0, dlp) if t is not None else zero
    with np.errstate(invalid="ignore"):
        lp = z.astype(np.float64) * scale - lse[:, None]
        p = np.where(np.isnan(lp), 0.0, np.exp(lp))
        a = np.where(p > 0, np.abs(lp), 0.0)
    ep = p * (2 * U * (a + np.abs(lse[:, None]) * (p > 0)) + 2.0 ** -22 + 3 * U)
    h = np.zeros(len(z)) if ent is None else np.abs(ent)
    size = (dl + dlp + dh * h)[:, None] + dh[:, None] * a
    slack = scale * (ep * size + p * (6 * U * size + dh[:, None] * 2 * U * (a + np.abs(lse[:, None]))))
    slack[np.arange(len(z)), np.maximum(t, 0) if t is not None else 0] += scale * 3 * U * dlp
    return HALF[dt] * (np.abs(ref) + slack) + slack + TINY[dt]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["plain", "masked"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradient(shape, kind, dt):
    torch = torch_cuda()
    z, t = _case(shape, dt, kind, 1)
    T, V, pad = shape
    r = _rng(2)
    zd, td = _dev(z, dt, pad), _i64(t)
    scale = np.float64(np.float32(0.7))
    f = cf.stitch_logprobs(zd, td, scale=0.7)
    lse, ent = _host(f[1]), _host(f[2])
    g = [r.standard_normal(T).astype(np.float32) for _ in range(3)]
    for use in ((1, 0, 0), (0, 1, 0), (1, 0, 1), (1, 1, 1)):
        dlp, dl, dh = (v if u else None for u, v in zip(use, g))
        tt = t if use[0] else None
        kw = dict(dlse=None if dl is None else _dev(dl), scale=0.7)
        if use[2]:
            kw.update(entropy=f[2], dentropy=_dev(dh))
        args = (td if use[0] else None, f[1], _dev(dlp) if use[0] else None)
        out = torch.full((T, V + 3), 9.0, dtype=zd.dtype, device="cuda")[:, :V]
        d = cf.stitch_logprobs_grad(zd, *args, **kw)
        k = slice(0, T, max(1, z.size >> 21))
        part = [None if v is None else v[k] for v in (tt, dlp, dl, dh)]
        ref = oracle.logprobs_grad(z[k], part[0], dlogprob=part[1], dlse=part[2], dentropy=part[3], scale=scale,
                                   lse=lse[k], entropy=ent[k])
        _within(d[k], ref, _grad_bound(z[k], part[0], scale, lse[k], ent[k] if use[2] else None, *part[1:], dt, ref),
                str(use))
        # rows apart, and in place
        cf.stitch_logprobs_grad(zd, *args, **kw, out=out)
        assert torch.equal(out, d) and (out._base[:, V:] == 9.0).all()
        own = zd.clone() if not pad else _dev(z, dt, pad)
        cf.stitch_logprobs_grad(own, *args, **kw, out=own)
        assert torch.equal(own, d) and (not pad or (own._base[:, V:] == 3.0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_gradient_ends(dt):
    """Masked tokens have none, a row without tokens zeros, a row with a NaN NaNs, the other rows their own."""
    z, t = _ends(dt, 1003)
    f = cf.stitch_logprobs(_dev(z, dt), _i64(t))
    one = np.ones(12, np.float32)
    d = _host(cf.stitch_logprobs_grad(_dev(z, dt), _i64(t), f[1], _dev(one), entropy=f[2], dentropy=_dev(one)))
    lse, ent = _host(f[1]), _host(f[2])
    ref = oracle.logprobs_grad(z, t, dlogprob=one, dentropy=one, lse=lse, entropy=ent)
    assert not d[0].any() and np.isnan(d[[4, 5, 11]]).all()
    rows = [3, 6, 7, 8, 9, 10]
    bound = _grad_bound(z[rows], t[rows], 1.0, lse[rows], ent[rows], one[rows], None, one[rows], dt, ref[rows])
    assert (np.abs(d[rows] - ref[rows]) <= bound).all()
    assert not d[3, :-1].any()


def test_rows_past_32_bits():
    """Rows behind the first 2^31 elements of the logits."""
    torch = torch_cuda()
    T, V = 34000, 65536
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("too little device memory")
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    rows = [0, 32767, 32768, 33999]
    small = _round(_rng(3).standard_normal((4, V)) * 2, "bf16")
    z[rows] = _dev(small, "bf16")
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    got = cf.stitch_logprobs(z, t, top=4)
    _check([g[rows] for g in got], small, np.zeros(4, np.int64), 1.0, 4)
    flat = _host(got[1][[1, 32766, 33998]])
    assert np.abs(flat - np.log(V)).max() < 1e-4
    d = torch.empty_like(z)
    cf.stitch_logprobs_grad(z, t, got[1], torch.ones(T, device="cuda"), out=d)
    ref = oracle.logprobs_grad(small, np.zeros(4, np.int64), dlogprob=np.ones(4), lse=_host(got[1][rows]))
    err = np.abs(_host(d[rows]) - ref)
    assert (err <= HALF["bf16"] * np.abs(ref) + 1e-5 * np.abs(ref) + 1e-12).all()


def test_wrapper_refusals():
    torch = torch_cuda()
    x, t = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    v = torch.zeros(4, device="cuda")
    for f, match in ((lambda: cf.stitch_logprobs(x, t.int()), "targets"),
                     (lambda: cf.stitch_logprobs(x, t[:3]), "targets"),
                     (lambda: cf.stitch_logprobs(x, t, top=33), "top"),
                     (lambda: cf.stitch_logprobs(x[:, :3], t, top=4), "top"),
                     (lambda: cf.stitch_logprobs(x, t, scale=0.0), "scale"),
                     (lambda: cf.stitch_logprobs(x.t(), t), "contiguous"),
                     (lambda: cf.stitch_logprobs(x[:, ::2], t), "contiguous"),
                     (lambda: cf.stitch_logprobs(x.double(), t), "dtype"),
                     (lambda: cf.stitch_logprobs(x[0], t), "dimensions"),
                     (lambda: cf.stitch_logprobs(x[:, :0], t), "columns"),
                     (lambda: cf.stitch_logprobs_grad(x, t, v), "targets"),
                     (lambda: cf.stitch_logprobs_grad(x, None, v), "gradient"),
                     (lambda: cf.stitch_logprobs_grad(x, t, v, v, dentropy=v), "entropy"),
                     (lambda: cf.stitch_logprobs_grad(x, t, v, v, out=x.half()), "out"),
                     (lambda: cf.stitch_logprobs_grad(x, t, v, v, out=x.expand(4, 64).t()[:4]), "out")):
        with pytest.raises(ValueError, match=match):
            f()
    assert cf.stitch_logprobs(x[:0], t[:0], top=3)[4].shape == (0, 3)
    assert cf.stitch_logprobs_grad(x[:, :0], t, v, v).shape == (4, 0)
