"""GPU parity of the grouped GEMM (forward, input gradient, weight gradient)
and of the low-rank adapter projection against the fp64 oracle, through the C
ABI and the torch-level calls.

Tolerance, element by element: half a step of the 16-bit output (at least
half its smallest subnormal), plus the fp32 accumulation.  A sum of n products
in any order is off by at most n 2^-23 sum|a b| (each addition loses at most
one fp32 step, truncation included, of a partial sum no larger than
sum|a b|); sum|a b| is the oracle's product of the absolute values.  GELU and
its slope: |slope| <= 1.13 carries the product's error, and the functions' own
(ex2.approx of an argument rounded to fp32) stays below 2^-16 of the value
while the exponent's argument is below 64, that is for |z| < 7; beyond, the
value is z or below 1e-10."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf, inputs
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8 / 1, "fp16": 2.0 ** -11}
TINY = {"bf16": 1e-38, "fp16": 2.0 ** -25}
ACC = 2.0 ** -23


def _round(a, dt):
    a = np.asarray(a, dtype=np.float32)
    return inputs.round_to_bf16(a) if dt == "bf16" else a.astype(np.float16).astype(np.float32)


def _dev(a, dt):
    torch = torch_cuda()
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16 if dt == "bf16" else torch.float16)


def _i32(a):
    torch = torch_cuda()
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _offsets(sizes, before=0):
    return np.concatenate([[before], before + np.cumsum(sizes)]).astype(np.int64)


def _check(got, ref, slack, dt, what):
    bound = HALF[dt] * np.abs(ref) + slack + TINY[dt]
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), f"{what}: non-finite"
    if err.size:
        worst = np.argmax(err - bound)
        assert err.flat[worst] <= bound.flat[worst], (
            f"{what}: {err.flat[worst]:.3e} > {bound.flat[worst]:.3e} at {np.unravel_index(worst, err.shape)}, "
            f"ref {ref.flat[worst]:.4f}")


def _status(ws):
    st, info = cf.cf_get_device_status(ws)
    assert st == cf.CF_OK, (cf.status_string(st), hex(info))


SENTINEL = 7.0  # what rows of no group hold before and after

# sizes, rows before the first and behind the last group, K, N
SHAPES = [
    ([1], 0, 0, 64, 128),
    ([2, 0, 1], 0, 0, 64, 64),
    ([0, 0, 5, 0], 3, 4, 136, 200),
    ([17, 16, 15, 1, 33], 0, 9, 72, 136),
    ([100, 0, 257, 31, 64], 5, 0, 200, 264),
    ([513, 40], 0, 1, 320, 520),
    ([3] * 40, 0, 0, 256, 72),
    ([1, 700, 2], 1, 1, 8, 8),
    ([300, 300, 300], 0, 0, 1024, 384),
    ([70, 33, 300], 0, 0, 192, 448),
]
IDS = [f"{len(s[0])}g{sum(s[0])}r{s[3]}x{s[4]}" for s in SHAPES]


# automatic, and forced: narrow and wide tiles, a shallow ring, few CTAs (several tiles each), CTA pairs
TUNINGS = {"auto": {}, "n16": dict(n_slice=16), "n64": dict(n_slice=64, cluster_m=1, stages=2), "n256": dict(n_slice=256, cluster_m=1, max_clusters=3),
           "pair128": dict(n_slice=128, cluster_m=2, max_clusters=2), "pair256": dict(n_slice=256, cluster_m=2, stages=3)}


def _tuning(name):
    return cf.tuning(**TUNINGS[name]) if TUNINGS[name] else None


def _forward_case(shape, dt, seed=0):
    sizes, before, behind, K, N = shape
    rng = _rng(seed + K + N)
    T = before + sum(sizes) + behind
    X = _round(rng.standard_normal((T, K)), dt)
    W = _round(rng.standard_normal((len(sizes), K, N)) * K ** -0.5, dt)
    return X, W, _offsets(sizes, before), T, K, N


def _gelu_slack(ref, z_slack):
    return 1.13 * z_slack + 2.0 ** -16 * np.abs(ref) + 1e-10


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("tun", TUNINGS)
def test_forward(shape, dt, act, tun):
    torch = torch_cuda()
    X, W, off, T, K, N = _forward_case(shape, dt)
    Xd = _dev(X, dt)
    out = torch.full((T, N), SENTINEL, dtype=Xd.dtype, device="cuda")
    z = torch.full((T, N), SENTINEL, dtype=Xd.dtype, device="cuda")
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, N, K, W.shape[0]))
    cf.grouped_gemm(Xd, _dev(W, dt), _i32(off), act=act, preact=z, out=out, workspace=ws, tuning=_tuning(tun))
    _status(ws)
    Y, Z = oracle.grouped_gemm(X, W, off, act=act)
    mag = oracle.grouped_gemm(np.abs(X), np.abs(W), off)[0]
    live = slice(off[0], off[-1])
    zs = K * ACC * mag[live]
    _check(_host(z)[live], Z[live], zs, dt, "Z")
    _check(_host(out)[live], Y[live], zs if act == "none" else _gelu_slack(Y[live], zs), dt, "Y")
    for t in (out, z):
        rest = np.delete(_host(t), np.arange(off[0], off[-1]), axis=0)
        assert np.all(rest == SENTINEL), "rows of no group were written"
    # without the pre-activation the output is the same bits
    out2 = torch.full((T, N), SENTINEL, dtype=Xd.dtype, device="cuda")
    cf.grouped_gemm(Xd, _dev(W, dt), _i32(off), act=act, out=out2, workspace=ws, tuning=_tuning(tun))
    assert torch.equal(out, out2)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("tun", TUNINGS)
def test_dgrad(shape, dt, act, tun):
    torch = torch_cuda()
    sizes, before, behind, K, N = shape
    X, W, off, T, K, N = _forward_case(shape, dt, seed=1)
    rng = _rng(2)
    dY = _round(rng.standard_normal((T, N)), dt)
    Z = _round(2.0 * rng.standard_normal((T, K)), dt) if act != "none" else None
    out = torch.full((T, K), SENTINEL, dtype=_dev([0.0], dt).dtype, device="cuda")
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, N, K, W.shape[0]))
    zd = _dev(Z, dt) if Z is not None else None
    cf.grouped_gemm_dgrad(_dev(dY, dt), _dev(W, dt), _i32(off), preact=zd, out=out, workspace=ws,
                          tuning=_tuning(tun))
    _status(ws)
    ref = oracle.grouped_gemm_dgrad(dY, W, off, preact=Z)
    plain = np.abs(oracle.grouped_gemm_dgrad(dY, W, off))
    slack = N * ACC * oracle.grouped_gemm_dgrad(np.abs(dY), np.abs(W), off)
    if Z is not None:
        slack = 1.13 * slack + 2.0 ** -16 * plain
    live = slice(off[0], off[-1])
    _check(_host(out)[live], ref[live], slack[live], dt, "dX")
    assert np.all(np.delete(_host(out), np.arange(off[0], off[-1]), axis=0) == SENTINEL)
    if zd is not None:  # in place of the pre-activation
        out_rows = out[off[0]:off[-1]].clone()
        cf.grouped_gemm_dgrad(_dev(dY, dt), _dev(W, dt), _i32(off), preact=zd, out=zd, workspace=ws,
                              tuning=_tuning(tun))
        assert torch.equal(zd[off[0]:off[-1]], out_rows)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("tun", [t for t in TUNINGS if t != "n16"])
def test_wgrad(shape, dt, tun):
    torch = torch_cuda()
    sizes, before, behind, K, N = shape
    rng = _rng(3)
    off = _offsets(sizes, before)
    T = before + sum(sizes) + behind
    X, dY = _round(rng.standard_normal((T, K)), dt), _round(0.1 * rng.standard_normal((T, N)), dt)
    # rows of no group hold what must not take part
    for a in (X, dY):
        a[:before] = np.nan
        a[off[-1]:] = np.inf
    out = torch.full((len(sizes), K, N), SENTINEL, dtype=_dev([0.0], dt).dtype, device="cuda")
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, N, K, len(sizes)))
    cf.grouped_gemm_wgrad(_dev(X, dt), _dev(dY, dt), _i32(off), out=out, workspace=ws, tuning=_tuning(tun))
    _status(ws)
    ref = oracle.grouped_gemm_wgrad(X, dY, off)
    mag = oracle.grouped_gemm_wgrad(np.abs(X), np.abs(dY), off)
    n = np.array(sizes, dtype=np.float64)[:, None, None]
    _check(_host(out), ref, n * ACC * mag, dt, "dW")


@pytest.mark.parametrize("direction", ["forward", "dgrad", "wgrad"])
@pytest.mark.parametrize("tun", TUNINGS)
def test_nan_stays_in_its_group(direction, tun):
    if direction == "wgrad" and tun == "n16":
        pytest.skip("refused: 64 columns at least")
    """One group's rows and weights are NaN: the other groups' results are the same bits as without."""
    torch = torch_cuda()
    shape = ([20, 37, 5, 70], 0, 0, 136, 264)
    X, W, off, T, K, N = _forward_case(shape, "bf16", seed=4)
    dY = _round(_rng(5).standard_normal((T, N)), "bf16")

    def run(x, dy, w):
        if direction == "forward":
            return cf.grouped_gemm(_dev(x, "bf16"), _dev(w, "bf16"), _i32(off), tuning=_tuning(tun))
        if direction == "dgrad":
            return cf.grouped_gemm_dgrad(_dev(dy, "bf16"), _dev(w, "bf16"), _i32(off), tuning=_tuning(tun))
        return cf.grouped_gemm_wgrad(_dev(x, "bf16"), _dev(dy, "bf16"), _i32(off), tuning=_tuning(tun))

    clean = run(X, dY, W)
    bad = 2
    Xn, Dn, Wn = X.copy(), dY.copy(), W.copy()
    Xn[off[bad]:off[bad + 1]] = np.nan
    Dn[off[bad]:off[bad + 1]] = np.inf
    Wn[bad] = np.nan
    dirty = run(Xn, Dn, Wn)
    if direction == "wgrad":
        keep = [e for e in range(4) if e != bad]
        assert torch.equal(clean[keep], dirty[keep]) and not torch.isfinite(dirty[bad]).any()
    else:
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[off[bad]:off[bad + 1]] = False
        assert torch.equal(clean[keep], dirty[keep]) and not torch.isfinite(dirty[~keep]).any()


LORA_SHAPES = [
    # sizes, before, behind, K, N, L, R, adapters
    ([1], 0, 0, 64, 128, 1, 8, [0]),
    ([1, 1, 1], 0, 0, 128, 64, 2, 16, [1, -1, 0]),
    ([1] * 64, 0, 0, 256, 384, 9, 16, None),
    ([0, 40, 0, 1, 7], 2, 3, 200, 136, 4, 24, [0, 3, 1, -1, 3]),
    ([300, 1, 64, 2], 0, 0, 320, 520, 3, 64, [2, 0, -1, 2]),
    ([5, 290], 1, 0, 72, 264, 2, 128, [1, 0]),
    ([33], 0, 0, 128, 128, 5, 40, [-1]),
    ([64, 63, 1, 200, 64, 5, 5], 0, 0, 136, 264, 3, 40, [0, 1, 2, -1, 2, 0, 1]),  # long and short requests in turn
    ([1] * 33 + [70] + [2] * 40, 0, 1, 1032, 192, 8, 72, None),
    ([3, 1, 2, 1, 1], 0, 0, 4096, 128, 4, 16, [3, 0, -1, 1, 0]),  # a divided contraction
]


def _lora_case(shape, dt, seed=6):
    sizes, before, behind, K, N, L, R, adapters = shape
    rng = _rng(seed)
    T = before + sum(sizes) + behind
    ad = np.array(adapters if adapters is not None else rng.integers(-1, L, len(sizes)))
    return dict(X=_round(rng.standard_normal((T, K)), dt), W=_round(rng.standard_normal((K, N)) * K ** -0.5, dt),
                bias=(0.1 * rng.standard_normal(N)).astype(np.float32),
                A=_round(rng.standard_normal((L, K, R)) * K ** -0.5, dt),
                B=_round(rng.standard_normal((L, R, N)) * R ** -0.5, dt), off=_offsets(sizes, before), ad=ad,
                scale=rng.uniform(0.5, 2.0, L).astype(np.float32), T=T, K=K, N=N, R=R)


def _lora_run(c, dt, bias=True, scale=True, **kw):
    torch = torch_cuda()
    X = _dev(c["X"], dt)
    out = torch.full((c["T"], c["N"]), SENTINEL, dtype=X.dtype, device="cuda")
    ws = cf.new_workspace(cf.cf_gemm_lora_workspace_size(c["T"], c["N"], c["K"], len(c["ad"]), c["R"]))
    cf.gemm_lora(X, _dev(c["W"], dt), torch.from_numpy(c["bias"]).cuda() if bias else None, _dev(c["A"], dt),
                 _dev(c["B"], dt), _i32(c["off"]), _i32(c["ad"]),
                 scale=torch.from_numpy(c["scale"]).cuda() if scale else None, out=out, workspace=ws, **kw)
    _status(ws)
    return out


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", LORA_SHAPES, ids=[f"{len(s[0])}s{sum(s[0])}r{s[3]}x{s[4]}R{s[6]}" for s in LORA_SHAPES])
@pytest.mark.parametrize("extras", [True, False])
@pytest.mark.parametrize("tun", TUNINGS)
def test_lora(shape, dt, extras, tun):
    c = _lora_case(shape, dt)
    out = _host(_lora_run(c, dt, extras, extras, tuning=_tuning(tun)))
    bias, scale = (c["bias"], c["scale"]) if extras else (None, None)
    ref = oracle.gemm_lora(c["X"], c["W"], bias, c["A"], c["B"], c["off"], c["ad"], scale)
    ab = {k: np.abs(c[k]) for k in ("X", "W", "A", "B")}
    zero = np.zeros_like(c["W"])
    shared = oracle.gemm_lora(ab["X"], ab["W"], np.abs(c["bias"]), ab["A"], ab["B"], c["off"], np.full(len(c["ad"]), -1))
    low = oracle.gemm_lora(ab["X"], zero, None, ab["A"], ab["B"], c["off"], c["ad"], scale)
    # H is held as two 16-bit parts, the rounded H and the rounded rest.  Each rounding is off by half a step at most,
    # u = 2^-8 (bf16) or 2^-11 (fp16) of the value, so H is off by u^2 of itself; and in fp16 by half the smallest
    # subnormal, 2^-25, at least
    parts = {"bf16": 2.0 ** -16, "fp16": 2.0 ** -22}[dt]
    slack = ACC * ((c["K"] + 2) * shared + (c["K"] + c["R"] + 2) * low) + parts * low
    if dt == "fp16":
        slack += 2.0 ** -25 * c["R"] * ab["B"].max()
    live = slice(c["off"][0], c["off"][-1])
    _check(out[live], ref[live], slack[live], dt, "Y")
    assert np.all(np.delete(out, np.arange(c["off"][0], c["off"][-1]), axis=0) == SENTINEL)


def test_lora_nan_stays_with_its_requests():
    torch = torch_cuda()
    c = _lora_case(([3, 1, 1, 40, 2], 0, 0, 128, 264, 3, 16, [0, 1, 2, 1, 0]), "bf16")
    clean = _lora_run(c, "bf16")
    for name in ("A", "B"):
        d = dict(c, **{name: c[name].copy()})
        d[name][1] = np.nan
        dirty = _lora_run(d, "bf16")
        hit = np.zeros(c["T"], bool)
        for s in (1, 3):
            hit[c["off"][s]:c["off"][s + 1]] = True
        hit = torch.from_numpy(hit).cuda()
        assert torch.equal(clean[~hit], dirty[~hit]) and torch.isnan(dirty[hit]).all()


def test_lora_without_adapters():
    """L = 0: the projection alone."""
    torch = torch_cuda()
    c = _lora_case(([5, 2], 0, 0, 64, 128, 1, 16, [-1, -1]), "bf16")
    full = _lora_run(c, "bf16")
    X = _dev(c["X"], "bf16")
    y = cf.gemm_lora(X, _dev(c["W"], "bf16"), torch.from_numpy(c["bias"]).cuda(), X.new_empty(0, 64, 16),
                     X.new_empty(0, 16, 128), _i32(c["off"]), _i32(c["ad"]))
    assert torch.equal(full, y)


def test_no_rows():
    torch = torch_cuda()
    W = torch.zeros(2, 64, 128, dtype=torch.bfloat16, device="cuda")
    off = _i32([0, 0, 0])
    X = W.new_empty(0, 64)
    assert cf.grouped_gemm(X, W, off).shape == (0, 128)
    assert cf.grouped_gemm_dgrad(W.new_empty(0, 128), W, off).shape == (0, 64)
    dw = cf.grouped_gemm_wgrad(X, W.new_empty(0, 128), off, out=torch.ones_like(W))
    assert not dw.any()
    # rows, but none in a group
    X = torch.full((9, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = cf.grouped_gemm(X, W, off, out=torch.full((9, 128), SENTINEL, dtype=torch.bfloat16, device="cuda"))
    assert torch.all(y == SENTINEL)
    assert not cf.grouped_gemm_wgrad(X, X.new_zeros(9, 128), off, out=torch.ones_like(W)).any()


@pytest.mark.parametrize("offsets", [[0, 9, 5, 12], [-3, 4, 8, 12], [0, 4, 8, 99], [2 ** 31 - 1, -2 ** 31, 0, 5]])
def test_bad_offsets_are_clamped_and_reported(offsets):
    """Offsets are clamped to [0, T] and to their running maximum, so no access leaves an array."""
    torch = torch_cuda()
    T, K, N = 12, 64, 128
    X = torch.ones(T, K, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(3, K, N, dtype=torch.bfloat16, device="cuda")
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, N, K, 3))
    fixed = np.maximum.accumulate(np.clip(np.array(offsets, dtype=np.int64), 0, T))
    y = cf.grouped_gemm(X, W, _i32(offsets), workspace=ws, out=torch.zeros(T, N, dtype=X.dtype, device="cuda"))
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_BOUNDS
    want = torch.zeros_like(y)
    want[fixed[0]:fixed[-1]] = K
    assert torch.equal(y, want)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK


def test_bad_adapters_are_none_and_reported():
    torch = torch_cuda()
    c = _lora_case(([2, 3, 1], 0, 0, 64, 128, 2, 8, [0, -1, -1]), "bf16")
    good = _lora_run(c, "bf16")
    ws = cf.new_workspace(cf.cf_gemm_lora_workspace_size(c["T"], c["N"], c["K"], 3, 8))
    y = cf.gemm_lora(_dev(c["X"], "bf16"), _dev(c["W"], "bf16"), torch.from_numpy(c["bias"]).cuda(),
                     _dev(c["A"], "bf16"), _dev(c["B"], "bf16"), _i32(c["off"]), _i32([0, 2, -7]),
                     scale=torch.from_numpy(c["scale"]).cuda(), workspace=ws)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_BOUNDS
    assert torch.equal(good, y)


SPLIT = [  # few tiles, long contractions: the tiles' contractions are divided among CTAs
    ([2, 1], 0, 0, 4096, 128), ([1, 0, 40], 1, 2, 2056, 264), ([200, 7], 0, 0, 1992, 128), ([16], 0, 0, 8192, 8)]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", SPLIT, ids=[f"{sum(s[0])}r{s[3]}x{s[4]}" for s in SPLIT])
@pytest.mark.parametrize("tun", ["auto", "n256", "n16"])
def test_divided_contraction(shape, dt, tun):
    """forward over a long K, input gradient over a long N, weight gradient over many rows; twice on one workspace
    (its counters return to zero), equal bits."""
    torch = torch_cuda()
    X, W, off, T, K, N = _forward_case(shape, dt, seed=7)
    E = W.shape[0]
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, max(N, K), max(N, K), E))
    live = slice(off[0], off[-1])
    Xd, Wd, Wt = _dev(X, dt), _dev(W, dt), _dev(np.swapaxes(W, 1, 2), dt)
    ref, Z = oracle.grouped_gemm(X, W, off, act="gelu_tanh")
    mag = oracle.grouped_gemm(np.abs(X), np.abs(W), off)[0]
    kw = dict(workspace=ws, tuning=_tuning(tun))
    y = cf.grouped_gemm(Xd, Wd, _i32(off), act="gelu_tanh", **kw)
    _status(ws)
    _check(_host(y)[live], ref[live], _gelu_slack(ref[live], K * ACC * mag[live]), dt, "Y")
    pre = _dev(2.0 * _rng(8).standard_normal((T, N)), dt)
    dx = cf.grouped_gemm_dgrad(Xd, Wt, _i32(off), preact=pre, **kw)  # rows of length K, "features" N
    _status(ws)
    slope = oracle.gelu_tanh_slope(_host(pre))
    _check(_host(dx)[live], (Z * slope)[live], (1.13 * K * ACC * mag + 2.0 ** -16 * np.abs(Z))[live], dt, "dX")
    rows = _offsets([3 * K // 2, 0, 1], 1)
    A, D = _round(_rng(9).standard_normal((rows[-1] + 2, 72)), dt), _round(_rng(10).standard_normal((rows[-1] + 2, N)) / 64, dt)
    A[rows[-1]:] = np.nan
    if tun != "n16":
        ws2 = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(A.shape[0], N, 72, 3))
        dw = cf.grouped_gemm_wgrad(_dev(A, dt), _dev(D, dt), _i32(rows), workspace=ws2, tuning=_tuning(tun))
        _status(ws2)
        want, wmag = oracle.grouped_gemm_wgrad(A, D, rows), oracle.grouped_gemm_wgrad(np.abs(A), np.abs(D), rows)
        _check(_host(dw), want, np.diff(rows)[:, None, None] * ACC * wmag, dt, "dW")
        assert torch.equal(dw, cf.grouped_gemm_wgrad(_dev(A, dt), _dev(D, dt), _i32(rows), workspace=ws2,
                                                     tuning=_tuning(tun)))
    y2 = cf.grouped_gemm(Xd, Wd, _i32(off), act="gelu_tanh", **kw)
    assert torch.equal(y[live], y2[live])


def test_one_workspace_serves_calls_of_many_sizes():
    """Grouped and adapter calls of different sizes in turn on one workspace give what fresh ones give."""
    torch = torch_cuda()
    ws = cf.new_workspace(1 << 26)
    for _ in range(2):
        for shape in LORA_SHAPES[:4] + [([2, 1], 0, 0, 4096, 128, 2, 16, [1, 0])]:
            c = _lora_case(shape, "bf16")
            X, off = _dev(c["X"], "bf16"), _i32(c["off"])
            args = (X, _dev(c["W"], "bf16"), None, _dev(c["A"], "bf16"), _dev(c["B"], "bf16"), off, _i32(c["ad"]))
            live = slice(c["off"][0], c["off"][-1])
            assert torch.equal(cf.gemm_lora(*args, workspace=ws)[live], cf.gemm_lora(*args)[live])
            W = _dev(np.stack([c["W"]] * len(c["ad"])), "bf16")
            y, fresh = (cf.grouped_gemm(X, W, off, workspace=w) for w in (ws, None))
            assert torch.equal(y[live], fresh[live])
            assert torch.equal(cf.grouped_gemm_wgrad(X[live], y[live], off - off[0], workspace=ws),
                               cf.grouped_gemm_wgrad(X[live], y[live], off - off[0]))
    _status(ws)
