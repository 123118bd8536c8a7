"""The grouped GEMM and the low-rank adapters at the ends of their ranges: rows of a long request that share their last
tile with short ones, very long sums, the largest middle values, the activation's ends, sums that are exact.

Bounds are those of the other parity files (half a step of the 16-bit output plus the fp32 sums'), or equality where
every partial sum is a whole number that fp32 holds."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import SENTINEL, _check, _dev, _host, _i32, _lora_case, _lora_run, _rng, _tuning
from tests.test_gpu_grouped_adapters import _bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tun", ["auto", "n256", "pair128", "pair256"])
@pytest.mark.parametrize("own", [16, 31, 32, 33, 47, 48, 58, 95, 100, 127])
def test_a_long_request_shares_its_last_tile(own, tun, dt):
    """A long request and short ones behind it in one tile: its rows in whole steps of the MMA's columns on the tensor
    cores, those that are left and the short requests' on the CUDA cores, single CTAs (steps of 16) and pairs (32)."""
    c = _lora_case(([own, 1, 2, 1, own, 3], 0, 2, 264, 392, 4, 24, [0, 1, 2, -1, 3, 1]), dt, seed=90 + own)
    ref, slack = _bounds(c, dt, c["bias"], c["scale"])
    live = slice(c["off"][0], c["off"][-1])
    out = _host(_lora_run(c, dt, tuning=_tuning(tun)))
    _check(out[live], ref[live], slack[live], dt, "Y")
    assert np.all(out[c["off"][-1]:] == SENTINEL)


def test_pairs_of_two_streams():
    """CTA pairs with shallow rings and all of tensor memory, launched on two streams at once: an SM holds one of them,
    so neither waits for tensor memory that the other holds."""
    torch = torch_cuda()
    X, W = _dev(_rng(1).standard_normal((700, 256)), "bf16"), _dev(_rng(2).standard_normal((3, 256, 520)) / 16, "bf16")
    off, tuning = _i32([0, 300, 301, 700]), cf.tuning(n_slice=256, cluster_m=2, stages=2)
    want = cf.grouped_gemm(X, W, off, tuning=tuning)
    dw = cf.grouped_gemm_wgrad(X, want, off, tuning=tuning)
    torch.cuda.synchronize()
    jobs = []
    for _ in range(2):
        size = cf.cf_grouped_gemm_workspace_size(700, 520, 256, 3)
        jobs.append((torch.cuda.Stream(), cf.new_workspace(size), torch.zeros_like(want), torch.zeros_like(dw)))
    torch.cuda.synchronize()
    for _ in range(50):
        for s, ws, y, d in jobs:
            cf.grouped_gemm(X, W, off, out=y, workspace=ws, stream=s, tuning=tuning)
            cf.grouped_gemm_wgrad(X, y, off, out=d, workspace=ws, stream=s, tuning=tuning)
    torch.cuda.synchronize()
    for _, ws, y, d in jobs:
        assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
        assert torch.equal(y, want) and torch.equal(d, dw)


def _counted(rows, K, N, every):
    """X [rows, K] with a 1 in every `every`-th row of a column, at another row for each column, and `every` rows apart;
    dY [rows, N] with row r holding 1 + column.  dW[k, n] = (1 + n) * the ones of column k."""
    torch = torch_cuda()
    X = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    for k in range(K):
        X[(k * every) // K::every, k] = 1.0
    dY = torch.arange(1, N + 1, device="cuda").to(torch.bfloat16).expand(rows, N).contiguous()
    return X, dY


@pytest.mark.parametrize("rows", [2 ** 26 + 5, 2 ** 27])
def test_weight_gradient_of_very_many_rows(rows):
    """One group past 2^26 rows (2^20 blocks of the contraction) is divided among the SMs like a shorter one: the sum
    counts every marked row once, and no wait runs out."""
    torch = torch_cuda()
    K = N = 8
    every = 2 ** 21
    X, dY = _counted(rows, K, N, every)
    X[-1] = 64.0  # the last row
    off = _i32([0, rows])
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(rows, N, K, 1))
    dw = cf.grouped_gemm_wgrad(X, dY, off, workspace=ws)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
    ones = (X.float().sum(0)).double()  # whole numbers below 2^24
    want = ones[:, None] * torch.arange(1, N + 1, device="cuda").double()
    assert torch.equal(dw[0].double(), want.to(torch.bfloat16).double())


def test_a_long_sum_that_is_not_divided_is_waited_for():
    """A group of very many rows beside a thousand empty ones, more tiles than may be divided: the wait for an
    accumulator grows with what is summed in it."""
    torch = torch_cuda()
    rows, K, N, E = 2_000_003, 136, 136, 1024
    X, dY = _counted(rows, K, N, 2 ** 15)
    dY.clamp_(max=8.0)
    off = _i32([0] * 500 + [rows] * (E + 1 - 500))
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(rows, N, K, E))
    dw = cf.grouped_gemm_wgrad(X, dY, off, workspace=ws, tuning=cf.tuning(timeout_us=1000))
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
    want = X.float().sum(0).double()[:, None] * dY[0].double()
    assert torch.equal(dw[499].double(), want.to(torch.bfloat16).double())
    assert not dw[:499].any() and not dw[500:].any()


@pytest.mark.parametrize("sizes,K", [([3, 1], 64), ([2], 4096), ([40], 64), ([100, 2], 64), ([40], 8192)])
def test_middle_products_beyond_the_parts_are_reported(sizes, K):
    """fp16: a finite middle value beyond +-131,008 is reported, in short requests, tiles and divided ones; values up to
    it, infinities, and products of other rows with this adapter are not."""
    torch = torch_cuda()
    N, R, T = 64, 8, sum(sizes) + 1
    X = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    X[:, K // 2] = 1024.0
    X[-1] = 60000.0  # a request without an adapter, in the same tile
    W = torch.zeros(K, N, dtype=torch.float16, device="cuda")
    A = torch.zeros(5, K, R, dtype=torch.float16, device="cuda")
    for a, v in enumerate((100.0, 127.9375, 128.0, float("inf"), -1000.0)):
        A[a, K // 2, R - 1] = v
    B = torch.full((5, R, N), 2.0 ** -6, dtype=torch.float16, device="cuda")
    off = _i32(np.concatenate([[0], np.cumsum(sizes), [T]]))
    ws = cf.new_workspace(cf.cf_gemm_lora_workspace_size(T, N, K, len(sizes) + 1, R))
    for a, status in enumerate((cf.CF_OK, cf.CF_OK, cf.CF_ERR_DEVICE_BOUNDS, cf.CF_OK, cf.CF_ERR_DEVICE_BOUNDS)):
        cf.gemm_lora(X, W, None, A, B, off, _i32([a] * len(sizes) + [-1]), workspace=ws)
        assert cf.cf_get_device_status(ws)[0] == status, a


@pytest.mark.parametrize("sizes,K", [([3, 1], 64), ([40], 64), ([100, 2], 64), ([40], 8192)])
def test_middle_products_beyond_the_largest_bf16_are_finite(sizes, K):
    """bf16: a middle value between the largest bf16 and the largest fp32 number is held by the two parts like any other
    one (the upper part must not round to infinity)."""
    torch = torch_cuda()
    N, R, T = 64, 8, sum(sizes)
    top = torch.finfo(torch.bfloat16).max
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[:, 0], X[:, 1] = 1.0, 3 * 2.0 ** -10
    W = torch.zeros(K, N, dtype=torch.bfloat16, device="cuda")
    A = torch.zeros(2, K, R, dtype=torch.bfloat16, device="cuda")
    A[0, :2, 0], A[1, :2, 0] = top, -top
    B = torch.full((2, R, N), 2.0 ** -100, dtype=torch.bfloat16, device="cuda")
    off = _i32(np.concatenate([[0], np.cumsum(sizes)]))
    h = top * (1 + 3 * 2.0 ** -10)  # closer to the largest fp32 number than to the largest bf16 one
    assert top < h < torch.finfo(torch.float32).max
    for a in (0, 1):
        y = cf.gemm_lora(X, W, None, A, B, off, _i32([a] * len(sizes))).double()
        want = (h if a == 0 else -h) * 2.0 ** -100
        assert ((y - want).abs() <= 2.0 ** -8 * abs(want)).all(), (a, y[0, 0].item(), want)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handle(handle):
    """0 and 1 are the legacy default stream's handles: the call waits for what is on that stream and what is on it
    later waits for the call."""
    torch = torch_cuda()
    X, W = _dev(_rng(3).standard_normal((300, 256)), "bf16"), _dev(_rng(4).standard_normal((2, 256, 264)) / 16, "bf16")
    off = _i32([0, 120, 300])
    want = cf.grouped_gemm(X, W, off)
    x, a = torch.zeros_like(X), torch.randn(4096, 4096, device="cuda")
    out = torch.zeros_like(want)
    with cf._launch_on(X.device, handle):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    for _ in range(20):  # keeps the stream busy before the input is there
        a = a @ a * 1e-3
    x.copy_(X)
    cf.grouped_gemm(x, W, off, out=out, stream=handle)
    got = out.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_stream_of_another_device_is_refused():
    torch = torch_cuda()

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    X, W = _dev(np.ones((4, 64)), "bf16"), _dev(np.ones((1, 64, 64)), "bf16")
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        cf.grouped_gemm(X, W, _i32([0, 4]), stream=Stream())
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        cf.gemm_lora(X, W[0], None, X.new_zeros(1, 64, 8), X.new_zeros(1, 8, 64), _i32([0, 4]), _i32([0]),
                     stream=Stream())


ENDS = [0.0, 1e-3, 1.0, 3.0, 6.5, 7.0, 8.0, 10.0, 11.75, 12.0, 12.5, 13.0, 100.0, 1000.0, 3e4]


def _ends(dt):
    """Both signs of the activation's interesting arguments and the type's largest, as numbers of the type."""
    torch = torch_cuda()
    t = torch.bfloat16 if dt == "bf16" else torch.float16
    v = torch.tensor(ENDS + [torch.finfo(t).max], device="cuda").to(t)
    return torch.cat([v, -v]), torch.tensor([float("inf"), float("-inf"), float("nan")] + [1.0] * 5, device="cuda").to(t)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tun", ["auto", "n64", "pair128"])
@pytest.mark.parametrize("K,at", [(8, 0), (4096, 2047), (4096, 4095)])
def test_activation_ends_forward(K, at, tun, dt):
    """Products that are exactly the ends of the activation: in whole tiles and in ones whose contraction is divided."""
    torch = torch_cuda()
    finite, special = _ends(dt)
    z = torch.cat([finite, special])
    N, T = z.numel(), 21
    X = torch.zeros(T, K, dtype=z.dtype, device="cuda")
    X[:, at] = 1.0
    W = torch.zeros(2, K, N, dtype=z.dtype, device="cuda")
    W[0, at] = z
    pre = torch.full((T, N), SENTINEL, dtype=z.dtype, device="cuda")
    y = cf.grouped_gemm(X, W, _i32([0, 20, T]), act="gelu_tanh", preact=pre, tuning=_tuning(tun))
    assert torch.equal(pre[:20].nan_to_num(9.0), z.expand(20, N).nan_to_num(9.0)) and not pre[20].any() and not y[20].any()
    n = finite.numel()
    got, want = _host(y[:20, :n]), oracle.gelu_tanh(_host(finite))[None, :].repeat(20, 0)
    # the function's own error (see test_gpu_grouped): 2^-16 of the value, 1e-10 where the value is below that
    _check(got, want, 2.0 ** -16 * np.abs(want) + 1e-10, dt, "gelu")
    assert torch.all(y[:20, n] == float("inf"))
    assert y[:20, n + 1:n + 3].isnan().all()  # -inf times 0, as x (1 + tanh) / 2 is, and NaN


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tun", ["auto", "n64", "pair128"])
@pytest.mark.parametrize("N,at", [(8, 0), (4096, 2047), (4096, 4095)])
def test_activation_ends_gradient(N, at, tun, dt):
    """The slope at the ends of the activation, times an input gradient of exactly 1 or -3."""
    torch = torch_cuda()
    finite, special = _ends(dt)
    z = torch.cat([finite, special])
    K, T = z.numel(), 21
    dY = torch.zeros(T, N, dtype=z.dtype, device="cuda")
    dY[:, at] = 1.0
    dY[1, at] = -3.0
    W = torch.zeros(1, K, N, dtype=z.dtype, device="cuda")
    W[0, :, at] = 1.0
    dx = cf.grouped_gemm_dgrad(dY, W, _i32([0, T]), preact=z.expand(T, K).contiguous(), tuning=_tuning(tun))
    n = finite.numel()
    slope = oracle.gelu_tanh_slope(_host(finite))
    want = slope[None, :] * _host(dY[:, at:at + 1])
    # p and 2 z p (1 - p) u' are each off by 2^-16 of themselves at most, and 1e-10 where they are below that
    _check(_host(dx[:, :n]), want, 2.0 ** -16 * (np.abs(want) + 3.0) + 3e-10, dt, "slope")
    for r, g in ((0, 1.0), (1, -3.0)):  # the slope's limits, 1 and 0
        assert dx[r, n].item() == g and dx[r, n + 1].item() == 0.0 and dx[r, n + 2].isnan()


EXACT_TUNINGS = {"auto": {}, "n256": dict(n_slice=256, cluster_m=1), "n64x5": dict(n_slice=64, cluster_m=1, max_clusters=5),
                 "n64x37": dict(n_slice=64, cluster_m=1, max_clusters=37), "pair128": dict(n_slice=128, cluster_m=2)}


def _whole(seed, dt, *shape):
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.bfloat16 if dt == "bf16" else torch.float16)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tun", EXACT_TUNINGS)
@pytest.mark.parametrize("rows,long,short", [([2, 0, 1], 4096, 136), ([1, 40], 8200, 72), ([130], 5000, 264), ([20, 300], 1992, 128)])
def test_whole_numbers_are_summed_exactly(rows, long, short, tun, dt):
    """Operands of -2..2: every partial sum is a whole number below 2^24, so fp32 sums are exact in any order and the
    result is the exact sum rounded once.  A block lost or counted twice at the border of two pieces shows."""
    torch = torch_cuda()
    tuning = cf.tuning(**EXACT_TUNINGS[tun])
    E, T = len(rows), sum(rows)
    bounds = np.concatenate([[0], np.cumsum(rows)])
    off = _i32(bounds)
    X, W = _whole(1, dt, T, long), _whole(2, dt, E, long, short)
    want = torch.cat([X[a:b].double() @ W[e].double() for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])
    assert want.abs().max() < 2 ** 24
    assert torch.equal(cf.grouped_gemm(X, W, off, tuning=tuning), want.to(X.dtype))
    dx = cf.grouped_gemm_dgrad(X, W.transpose(1, 2).contiguous(), off, tuning=tuning)
    assert torch.equal(dx, want.to(X.dtype))
    # the weight gradient's long sum runs over rows: groups of `long` rows, one row, none, and the rest
    total = 3 * long
    A, D = _whole(3, dt, total, 72), _whole(4, dt, total, short)
    cuts = [0, long, long + 1, long + 1, total - 3]
    dw = cf.grouped_gemm_wgrad(A, D, _i32(cuts), tuning=tuning)
    want = torch.stack([A[a:b].double().T @ D[a:b].double() for a, b in zip(cuts, cuts[1:])])
    assert torch.equal(dw, want.to(A.dtype))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("tun", EXACT_TUNINGS)
@pytest.mark.parametrize("sizes,K,R", [([1], 4096, 16), ([1, 1, 3, 1], 8200, 24), ([40, 1, 2], 1992, 72), ([300, 2, 17, 64], 136, 8)])
def test_adapters_of_whole_numbers_are_exact(sizes, K, R, tun, dt):
    """The same for the adapters: the middle product is a whole number below 2^16, which its two parts hold."""
    torch = torch_cuda()
    S, T, N, L = len(sizes), sum(sizes), 264, 3
    bounds = np.concatenate([[0], np.cumsum(sizes)])
    X, W, A, B = _whole(5, dt, T, K), _whole(6, dt, K, N), _whole(7, dt, L, K, R), _whole(8, dt, L, R, N)
    bias, scale = _whole(9, dt, N).float(), torch.tensor([1.0, 2.0, -4.0], device="cuda")
    ad = [(i * 2 + 1) % (L + 1) - 1 for i in range(S)]
    y = cf.gemm_lora(X, W, bias, A, B, _i32(bounds), _i32(ad), scale=scale, tuning=cf.tuning(**EXACT_TUNINGS[tun]))
    want = X.double() @ W.double() + bias.double()
    for a, lo, hi in zip(ad, bounds, bounds[1:]):
        if a >= 0:
            h = scale[a].double() * (X[lo:hi].double() @ A[a].double())
            assert h.abs().max() < 2 ** 16
            want[lo:hi] += h @ B[a].double()
    assert want.abs().max() < 2 ** 24
    assert torch.equal(y, want.to(X.dtype))


@pytest.mark.parametrize("tun", [None, dict(n_slice=256, cluster_m=1), dict(n_slice=32)])
def test_the_most_rows(tun):
    """2^31 - 512 rows of 8 columns (34 GB each of X and Y) in two groups: rows from everywhere, and the ends."""
    torch = torch_cuda()
    T, K, N = 2 ** 31 - 512, 8, 8
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    cut = 2 ** 31 - 2 ** 21
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    pick = torch.cat([torch.randint(0, T, (4096,), device="cuda", generator=torch.Generator("cuda").manual_seed(1)),
                      torch.arange(300, device="cuda"), torch.arange(cut - 300, cut + 300, device="cuda"),
                      torch.arange(T - 300, T - 2, device="cuda")])
    X[pick] = torch.randint(-2, 3, (pick.numel(), K), device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(X.dtype)
    W = _whole(1, "bf16", 2, K, N)
    Y = torch.full((T, N), SENTINEL, dtype=X.dtype, device="cuda")
    ws = cf.new_workspace(cf.cf_grouped_gemm_workspace_size(T, N, K, 2))
    tuning = cf.tuning(**tun) if tun else None
    cf.grouped_gemm(X, W, _i32([0, cut, T - 2]), out=Y, workspace=ws, tuning=tuning)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
    want = torch.where((pick < cut)[:, None], X[pick].double() @ W[0].double(), X[pick].double() @ W[1].double())
    assert torch.equal(Y[pick].double(), want)
    assert (Y[T - 2:] == SENTINEL).all()
    rest = torch.randint(0, T - 2, (100_000,), device="cuda")  # nearly all of them rows of zeros
    assert torch.equal((Y[rest] != 0).any(1), (X[rest].float() @ W[0].float() != 0).any(1) & (rest < cut)
                       | (X[rest].float() @ W[1].float() != 0).any(1) & (rest >= cut))
    if tun is None:
        dw = cf.grouped_gemm_wgrad(X, Y, _i32([0, cut, T - 2]), workspace=ws)
        assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
        one = pick.unique()
        for e, rows in ((0, one[one < cut]), (1, one[(one >= cut) & (one < T - 2)])):
            want = X[rows].double().T @ Y[rows].double()
            assert want.abs().max() < 2 ** 24 and torch.equal(dw[e].double(), want.to(X.dtype).double())
