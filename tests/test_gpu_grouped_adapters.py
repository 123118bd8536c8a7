"""Low-rank adapters over requests of every length in one batch: long ones
with tiles of their own, runs of short ones that join them or stand alone,
neighbours that share an adapter, empty ones between; a NaN in an adapter or
a row stays with its requests; the ends of the middle product's range."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import (ACC, SENTINEL, TUNINGS, _check, _dev, _host, _i32, _lora_case, _lora_run, _rng,
                                    _status, _tuning)

pytestmark = pytest.mark.gpu

MIXED = [17, 1, 1, 33, 2, 0, 15, 64, 31, 1, 130, 5, 0, 16, 3, 300, 1, 1, 1, 0]
CASES = [  # sizes, before, behind, K, N, L, R, adapters
    (MIXED, 0, 0, 136, 264, 3, 8, None),
    (MIXED, 2, 3, 320, 392, 4, 72, None),
    (MIXED, 0, 1, 4104, 2064, 5, 8, None),
    ([17, 1, 100, 120, 3, 40, 0, 2], 1, 2, 8192, 4096, 3, 8, None),
    ([40, 1, 1, 30, 7, 2, 2, 90, 1], 0, 0, 264, 136, 3, 24, [1, 1, 1, 1, 1, 2, 2, 2, 2]),  # neighbours that share
    ([1, 2, 3, 4, 5, 0, 6], 0, 0, 264, 136, 2, 24, [1, 1, 1, 1, 1, 0, 1]),
    ([20, 3, 0, 50, 1], 0, 0, 264, 136, 2, 24, [-1, -1, 1, -1, -1]),
    ([200] + [1] * 40, 0, 0, 136, 264, 7, 16, None),  # a run longer than what joins
]


def _bounds(c, dt, bias, scale):
    """Oracle and what fp32 sums in any order and the middle product's two 16-bit parts may add to it.

    H = up + rest, up the rounded H and rest the rounded difference: each rounding is off by half a step at most, u of
    the value with u = 2^-8 (bf16) or 2^-11 (fp16), so H is off by u^2 of itself: 2^-16 and 2^-22; and in fp16 by half
    the smallest subnormal, 2^-25, where the rest falls below the normal range."""
    ref = oracle.gemm_lora(c["X"], c["W"], bias, c["A"], c["B"], c["off"], c["ad"], scale)
    ab = {k: np.abs(c[k]) for k in ("X", "W", "A", "B")}
    none = np.full(len(c["ad"]), -1)
    shared = oracle.gemm_lora(ab["X"], ab["W"], np.abs(c["bias"]), ab["A"], ab["B"], c["off"], none)
    low = oracle.gemm_lora(ab["X"], np.zeros_like(c["W"]), None, ab["A"], ab["B"], c["off"], c["ad"], scale)
    slack = ACC * ((c["K"] + 2) * shared + (c["K"] + c["R"] + 2) * low) + {"bf16": 2.0 ** -16, "fp16": 2.0 ** -22}[dt] * low
    if dt == "fp16":
        slack = slack + 2.0 ** -25 * c["R"] * ab["B"].max()
    return ref, slack


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_requests_of_every_length(case, dt):
    torch = torch_cuda()
    c = _lora_case(CASES[case], dt, seed=30 + case)
    ref, slack = _bounds(c, dt, c["bias"], c["scale"])
    live = slice(c["off"][0], c["off"][-1])
    for tun in TUNINGS:
        first = _lora_run(c, dt, tuning=_tuning(tun))
        out = _host(first)
        _check(out[live], ref[live], slack[live], dt, f"Y, {tun}")
        assert np.all(np.delete(out, np.arange(c["off"][0], c["off"][-1]), axis=0) == SENTINEL)
        assert torch.equal(first, _lora_run(c, dt, tuning=_tuning(tun)))


@pytest.mark.parametrize("tun", TUNINGS)
@pytest.mark.parametrize("what", ["A", "B", "X"])
def test_nan_stays_with_its_requests(what, tun):
    """A NaN in one adapter reaches the rows of its own requests, one in a row of X that row; nothing else changes."""
    torch = torch_cuda()
    c = _lora_case(CASES[1], "bf16", seed=50)
    clean = _lora_run(c, "bf16", tuning=_tuning(tun))
    d = dict(c, **{what: c[what].copy()})
    hit = np.zeros(c["T"], bool)
    if what == "X":
        rows = [c["off"][s] for s in (1, 3, 8, 15)] + [c["off"][4] - 1]
        d["X"][rows] = np.nan
        hit[rows] = True
    else:
        d[what][1] = np.nan
        for s in np.flatnonzero(c["ad"] == 1):
            hit[c["off"][s]:c["off"][s + 1]] = True
        assert 0 < hit.sum() < c["T"] // 2
    dirty = _lora_run(d, "bf16", tuning=_tuning(tun))
    hit = torch.from_numpy(hit).cuda()
    assert torch.equal(clean[~hit], dirty[~hit]) and torch.isnan(dirty[hit]).all()


@pytest.mark.parametrize("sizes", [[3, 1], [40], [100, 2]])
def test_middle_product_beyond_fp16(sizes):
    """fp16 operands: a middle value up to 131,008 is held as the sum of two fp16 numbers, one beyond counts as that,
    an infinity stays one."""
    torch = torch_cuda()
    K, N, R = 64, 64, 8
    T, L = sum(sizes), 4
    X = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    X[:, 0] = 1000.0
    W = torch.zeros(K, N, dtype=torch.float16, device="cuda")
    A = torch.zeros(L, K, R, dtype=torch.float16, device="cuda")
    A[0, 0, 0], A[1, 0, 0], A[2, 0, 0], A[3, 0, 0] = 100.0, -125.0, 1000.0, float("inf")
    B = torch.full((L, R, N), 2.0 ** -6, dtype=torch.float16, device="cuda")
    off = _i32(np.concatenate([[0], np.cumsum(sizes)]))
    for a, want in enumerate((1e5 / 64, -125e3 / 64, 131008.0 / 64, float("inf"))):
        y = cf.gemm_lora(X, W, None, A, B, off, _i32([a] * len(sizes)))
        assert torch.all(y == torch.tensor(want, device="cuda").half()), (a, want)


@pytest.mark.parametrize("tun", TUNINGS)
def test_same_rows_same_bits_alone_and_in_a_batch_of_copies(tun):
    """Every request of a batch of equal one-row requests gets the same row, with its adapter and without."""
    torch = torch_cuda()
    c = _lora_case(([1] * 40, 0, 0, 264, 136, 2, 16, [0, 1] * 20), "bf16", seed=60)
    c["X"][:] = c["X"][0]
    y = _lora_run(c, "bf16", tuning=_tuning(tun))
    for a in (0, 1):
        assert torch.equal(y[a::2], y[a:a + 1].expand(20, -1))


def test_replayed_after_its_inputs_were_written():
    """A graph that writes offsets, adapters, bias, scale and X and then makes the call, back to back: every replay reads
    what its own copies wrote, although the call's second launch starts before its first has ended."""
    torch = torch_cuda()
    K, N, L, R, S, T = 264, 136, 3, 24, 20, 200
    rng = _rng(70)
    W, A, B = (torch.from_numpy(rng.standard_normal(n)).cuda().bfloat16() / 8 for n in ((K, N), (L, K, R), (L, R, N)))
    sets = []
    for _ in range(6):
        cuts = np.sort(rng.integers(0, T + 1, S - 1))
        sets.append((_i32(np.concatenate([[0], cuts, [T]])), _i32(rng.integers(-1, L, S)),
                     torch.from_numpy(rng.standard_normal(N)).cuda().float(),
                     torch.from_numpy(rng.uniform(0.5, 2.0, L)).cuda().float(),
                     torch.from_numpy(rng.standard_normal((T, K))).cuda().bfloat16()))
    off, ad, bias, scale, X = (t.clone() for t in sets[0])
    ws = cf.new_workspace(cf.cf_gemm_lora_workspace_size(T, N, K, S, R))
    src = [t.clone() for t in sets[0]]
    out = torch.empty(T, N, dtype=X.dtype, device="cuda")

    def step():
        for to, of in zip((off, ad, bias, scale, X), src):
            to.copy_(of)
        cf.gemm_lora(X, W, bias, A, B, off, ad, scale=scale, out=out, workspace=ws)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
            step()
        got = []
        for s in sets * 3:
            for to, of in zip(src, s):
                to.copy_(of)
            graph.replay()
            got.append(out.clone())
    torch.cuda.synchronize()
    for (o, a, b, sc, x), y in zip(sets * 3, got):
        assert torch.equal(y, cf.gemm_lora(x, W, b, A, B, o, a, scale=sc))
    _status(ws)


def test_workspace_of_another_kind_is_refused():
    torch = torch_cuda()
    X = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(2, 64, 128, dtype=torch.bfloat16, device="cuda")
    n = cf.cf_grouped_gemm_workspace_size(8, 128, 64, 2)
    for ws in (torch.zeros(n, dtype=torch.uint8), cf.new_workspace(2 * n)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            cf.grouped_gemm(X, W, _i32([0, 4, 8]), workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            cf.grouped_gemm(X, W, _i32([0, 4, 8]), workspace=ws, stream=torch.cuda.Stream())


@pytest.mark.parametrize("sizes", [[1, 1, 2], [40, 3, 200]])
def test_a_wait_that_runs_out_is_reported(sizes):
    """Both launches wait for an arrival that nobody makes: their roles drain, the status is a timeout, and after the
    workspace is zeroed the next call on it is right."""
    torch = torch_cuda()
    c = _lora_case((sizes, 0, 0, 264, 136, 2, 16, [i % 2 for i in range(len(sizes))]), "bf16", seed=80)
    args = (_dev(c["X"], "bf16"), _dev(c["W"], "bf16"), None, _dev(c["A"], "bf16"), _dev(c["B"], "bf16"),
            _i32(c["off"]), _i32(c["ad"]))
    n = cf.cf_gemm_lora_workspace_size(c["T"], c["N"], c["K"], len(sizes), c["R"])
    ws = cf.new_workspace(n)
    cf.gemm_lora(*args, workspace=ws, tuning=cf.tuning(extra_arrivals=1, timeout_us=2000))
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
    cf.cf_workspace_init(ws, n)
    assert torch.equal(cf.gemm_lora(*args, workspace=ws), cf.gemm_lora(*args))
    _status(ws)
