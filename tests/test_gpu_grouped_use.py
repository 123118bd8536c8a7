"""The grouped GEMM and the low-rank adapter projection as a program uses
them: together in a step of a mixture-of-experts layer and its gradient, on
other streams, captured into CUDA graphs and replayed with other group sizes,
chained with programmatic dependent launch on and off, beside the library's
other calls, from several threads, at many groups and past 2^31 elements."""
import threading

import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf, inputs
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu

T, D, F, E = 300, 128, 256, 5


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _bf16(*shape, std=1.0, seed=0):
    return inputs.round_to_bf16((_rng(seed).standard_normal(shape) * std).astype(np.float32))


def _dev(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.bfloat16)


def _i32(a):
    torch = torch_cuda()
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)])


def _layer(seed=1):
    """Rows sorted by expert, adapters on the projection before the experts, W1 [E, D, F], W2 [E, F, D]."""
    return dict(x=_bf16(T, D, seed=seed), wp=_bf16(D, D, std=D ** -0.5, seed=seed + 1),
                a=_bf16(3, D, 16, std=D ** -0.5, seed=seed + 2), b=_bf16(3, 16, D, std=0.25, seed=seed + 3),
                w1=_bf16(E, D, F, std=D ** -0.5, seed=seed + 4), w2=_bf16(E, F, D, std=F ** -0.5, seed=seed + 5),
                g=_bf16(T, D, seed=seed + 6), requests=_offsets([1, 1, 100, 70, 1, 127]),
                adapters=np.array([0, -1, 1, 2, 2, 0]), experts=_offsets([90, 0, 17, 150, 43]))


def _step(c, tuning=None, ws=None, to=_dev):
    """Adapted projection -> up with GELU -> down; then the gradients of both experts' weights and of their input."""
    torch = torch_cuda()
    d = {k: to(v) for k, v in c.items() if k not in ("requests", "adapters", "experts")}
    off = _i32(c["experts"])
    kw = dict(tuning=tuning, workspace=ws)
    p = cf.gemm_lora(d["x"], d["wp"], None, d["a"], d["b"], _i32(c["requests"]), _i32(c["adapters"]), **kw)
    z = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    h = cf.grouped_gemm(p, d["w1"], off, act="gelu_tanh", preact=z, **kw)
    y = cf.grouped_gemm(h, d["w2"], off, **kw)
    dw2 = cf.grouped_gemm_wgrad(h, d["g"], off, **kw)
    dz = cf.grouped_gemm_dgrad(d["g"], d["w2"], off, preact=z, **kw)
    dw1 = cf.grouped_gemm_wgrad(p, dz, off, **kw)
    dp = cf.grouped_gemm_dgrad(dz, d["w1"], off, **kw)
    return dict(p=p, z=z, h=h, y=y, dw2=dw2, dz=dz, dw1=dw1, dp=dp)


def _close(got, ref, steps, what):
    """Each stage is held to `steps` roundings of bf16 (2^-8 of the stage's scale each): its own, and those of the
    stages whose rounded outputs it takes, which the oracle rounds alike but fp32 sums may round the other way."""
    err = np.abs(got - ref).max()
    bound = steps * 2.0 ** -8 * np.abs(ref).max()
    assert err <= bound, f"{what}: {err:.3e} > {bound:.3e}"


def test_layer_and_its_gradient():
    c = _layer()
    o = {k: _host(v) for k, v in _step(c).items()}
    off, r = c["experts"], lambda a: inputs.round_to_bf16(a.astype(np.float32)).astype(np.float64)
    p = r(oracle.gemm_lora(c["x"], c["wp"], None, c["a"], c["b"], c["requests"], c["adapters"]))
    h, z = (r(v) for v in oracle.grouped_gemm(p, c["w1"], off, act="gelu_tanh"))
    y = oracle.grouped_gemm(h, c["w2"], off)[0]
    dz = r(oracle.grouped_gemm_dgrad(c["g"], c["w2"], off, preact=z))
    ref = dict(p=p, z=z, h=h, y=y, dw2=oracle.grouped_gemm_wgrad(h, c["g"], off), dz=dz,
               dw1=oracle.grouped_gemm_wgrad(p, dz, off), dp=oracle.grouped_gemm_dgrad(dz, c["w1"], off))
    for (k, want), steps in zip(ref.items(), (1, 2, 3, 4, 4, 4, 5, 5)):
        _close(o[k], want, steps, k)
    assert not o["dw1"][1].any() and not o["dw2"][1].any()


def test_chain_is_the_same_with_and_without_overlap_and_in_a_graph():
    """Every call reads its predecessor's output: with programmatic dependent launch, without, and replayed."""
    torch = torch_cuda()
    c = _layer(3)
    ws = cf.new_workspace(max(cf.cf_grouped_gemm_workspace_size(T, F, F, E),
                              cf.cf_gemm_lora_workspace_size(T, D, D, 6, 16)))
    plain = _step(c, cf.tuning(disable_pdl=1), ws)
    for _ in range(3):
        over = _step(c, None, ws)
        for k in plain:
            assert torch.equal(plain[k], over[k]), k
    held = {k: _dev(v) for k, v in c.items() if k not in ("requests", "adapters", "experts")}
    off, req, ad = _i32(c["experts"]), _i32(c["requests"]), _i32(c["adapters"])
    out = {k: torch.empty_like(v) for k, v in plain.items()}

    def run(s=None):
        kw = dict(workspace=ws, stream=s)
        cf.gemm_lora(held["x"], held["wp"], None, held["a"], held["b"], req, ad, out=out["p"], **kw)
        cf.grouped_gemm(out["p"], held["w1"], off, act="gelu_tanh", preact=out["z"], out=out["h"], **kw)
        cf.grouped_gemm(out["h"], held["w2"], off, out=out["y"], **kw)
        cf.grouped_gemm_wgrad(out["h"], held["g"], off, out=out["dw2"], **kw)
        cf.grouped_gemm_dgrad(held["g"], held["w2"], off, preact=out["z"], out=out["dz"], **kw)
        cf.grouped_gemm_wgrad(out["p"], out["dz"], off, out=out["dw1"], **kw)
        cf.grouped_gemm_dgrad(out["dz"], held["w1"], off, out=out["dp"], **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            run()
    for v in out.values():
        v.zero_()
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in plain:
        assert torch.equal(plain[k], out[k]), k
    # the sizes are read on the device: the same graph serves another batch
    other = dict(c, experts=_offsets([0, 130, 130, 0, 40]), requests=_offsets([64, 0, 1, 200, 30, 5]),
                 adapters=np.array([2, 1, 0, -1, 1, 0]))
    for t, k in ((off, "experts"), (req, "requests"), (ad, "adapters")):
        t.copy_(_i32(other[k]))
    graph.replay()
    torch.cuda.synchronize()
    want = _step(other, cf.tuning(disable_pdl=1))
    for k in want:
        assert torch.equal(want[k], out[k]), k
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK


def test_two_graphs_that_share_a_workspace():
    torch = torch_cuda()
    ws = cf.new_workspace(1 << 26)
    jobs = []
    for seed, sizes, K, N in ((1, [3, 1], 4096, 256), (2, [200, 0, 30], 136, 264)):
        X, W = _dev(_bf16(sum(sizes), K, seed=seed)), _dev(_bf16(len(sizes), K, N, std=K ** -0.5, seed=seed + 5))
        off = _i32(_offsets(sizes))
        out = torch.empty(sum(sizes), N, dtype=torch.bfloat16, device="cuda")
        want = cf.grouped_gemm(X, W, off)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                cf.grouped_gemm(X, W, off, out=out, workspace=ws)
        jobs.append((g, out, want, (X, W, off)))
    for _ in range(3):
        for g, out, want, _ in jobs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out, want, _ in jobs:
            assert torch.equal(out, want)


@pytest.mark.parametrize("handle", [False, True])
def test_other_streams(handle):
    """A stream object or its handle: inputs made on it are waited for, nothing runs on the current stream."""
    torch = torch_cuda()
    c = _layer(5)
    want = cf.grouped_gemm(_dev(c["x"]), _dev(c["w1"]), _i32(c["experts"]), act="gelu_tanh")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):  # keeps the stream busy before the input is there
            a = a @ a * 1e-3
        x = _dev(c["x"])
        w, off = _dev(c["w1"]), _i32(c["experts"])
    y = cf.grouped_gemm(x, w, off, act="gelu_tanh", stream=s.cuda_stream if handle else s)
    s.synchronize()
    assert torch.equal(y, want)


def test_threads():
    """Several threads, each on its own stream and workspace, at kernels and shared-memory sizes of all kinds."""
    torch = torch_cuda()
    c = _layer(7)
    want = _step(c)
    torch.cuda.synchronize()
    fails = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got = _step(c)
                s.synchronize()
            for k in want:
                if not torch.equal(got[k], want[k]):
                    fails.append(k)
        except Exception as ex:  # noqa: BLE001 -- reported below
            fails.append(repr(ex))

    th = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in th]
    [t.join() for t in th]
    assert not fails, fails


def test_beside_the_other_calls():
    """The adapted projection feeding the fused GEMM + LayerNorm and a stitched softmax's input, on one stream."""
    torch = torch_cuda()
    c = _layer(9)
    x, wp, a, b = (_dev(c[k]) for k in ("x", "wp", "a", "b"))
    req, ad = _i32(c["requests"]), _i32(c["adapters"])
    w, ones, zeros = _dev(_bf16(D, 256, std=D ** -0.5, seed=4)), torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
    p = cf.gemm_lora(x, wp, None, a, b, req, ad)
    torch.cuda.synchronize()
    want = cf.gemm_fused_rownorm(p, w, zeros, ones, zeros)
    torch.cuda.synchronize()
    for _ in range(5):
        p2 = cf.gemm_lora(x, wp, None, a, b, req, ad)
        got = cf.gemm_fused_rownorm(p2, w, zeros, ones, zeros)
        y = cf.grouped_gemm(got, _dev(_bf16(1, 256, 64, seed=8)), _i32([0, T]))
        assert torch.equal(p, p2) and torch.equal(want, got) and torch.isfinite(y).all()


def test_many_groups():
    """1024 groups of 0 to 3 rows, and as many requests."""
    torch = torch_cuda()
    sizes = _rng(11).integers(0, 4, 1024)
    off, K, N = _offsets(sizes), 72, 136
    X, W = _bf16(off[-1], K, seed=12), _bf16(1024, K, N, std=K ** -0.5, seed=13)
    got = _host(cf.grouped_gemm(_dev(X), _dev(W), _i32(off)))
    ref = oracle.grouped_gemm(X, W, off)[0]
    _close(got, ref, 1.01, "1024 groups")
    dw = _host(cf.grouped_gemm_wgrad(_dev(X), _dev(got.astype(np.float32)), _i32(off)))
    _close(dw, oracle.grouped_gemm_wgrad(X, got, off), 1.01, "1024 groups' weights")
    ad = _rng(14).integers(-1, 7, 1024)
    A, B = _bf16(7, K, 8, std=K ** -0.5, seed=15), _bf16(7, 8, N, std=0.3, seed=16)
    y = _host(cf.gemm_lora(_dev(X), _dev(W[0]), None, _dev(A), _dev(B), _i32(off), _i32(ad)))
    _close(y, oracle.gemm_lora(X, W[0], None, A, B, off, ad), 1.01, "1024 requests")


def test_rows_past_2_31_elements():
    """1.2 million rows of 2048 columns: 2.4 G elements of Y, of dX and of the adapters' Y; the rows at the end and
    at random against the oracle."""
    torch = torch_cuda()
    rows, K, N = 1_200_000, 64, 2048
    X = torch.randn(rows, K, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    W = _dev(_bf16(2, K, N, std=K ** -0.5, seed=17))
    off = [0, 700_001, rows - 3]
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    cf.grouped_gemm(X, W, _i32(off), out=y)
    pick = torch.tensor(sorted(set(_rng(18).integers(0, rows - 3, 200)) | {0, 700_000, 700_001, rows - 4}), device="cuda")
    Xh, Wh = _host(X[pick]), _host(W)
    e = (pick.cpu().numpy() >= 700_001).astype(int)
    ref = np.stack([x @ Wh[i] for x, i in zip(Xh, e)])
    _close(_host(y[pick]), ref, 1.01, "Y")
    assert not y[rows - 3:].any()
    # the input gradient with the roles of the lengths turned: rows of 64 from W^T
    dx = cf.grouped_gemm_dgrad(X, W.transpose(1, 2).contiguous(), _i32(off), out=y.zero_())
    _close(_host(dx[pick]), ref, 1.01, "dX")
    dw = cf.grouped_gemm_wgrad(X, y[:, :64].contiguous(), _i32(off))
    want = torch.stack([X[a:b].double().T @ y[a:b, :64].double() for a, b in zip(off[:-1], off[1:])])
    assert (dw.double() - want).abs().max() <= 2.0 ** -8 * 1.1 * want.abs().max()
    A, B = _dev(_bf16(2, K, 8, std=K ** -0.5, seed=19)), _dev(_bf16(2, 8, N, std=0.3, seed=20))
    cf.gemm_lora(X, W[0], None, A, B, _i32(off), _i32([1, 0]), out=y.zero_())
    Ah, Bh = _host(A), _host(B)
    ref = np.stack([x @ Wh[0] + (x @ Ah[1 - i]) @ Bh[1 - i] for x, i in zip(Xh, e)])
    _close(_host(y[pick]), ref, 1.01, "adapters' Y")
    assert not y[rows - 3:].any()


def test_weights_past_2_31_elements():
    """Three experts of 16384 x 65536: dW has 3.2 G elements, and the forward reads as many."""
    torch = torch_cuda()
    K, N, sizes = 16384, 65536, [20, 0, 33]
    off = _offsets(sizes)
    X, dY = _bf16(off[-1], K, seed=21), _bf16(off[-1], N, seed=22)
    dw = cf.grouped_gemm_wgrad(_dev(X), _dev(dY), _i32(off))
    assert not dw[1].any()
    for e in (0, 2):
        rows = slice(off[e], off[e + 1])
        for k, n in ((0, 0), (K - 40, N - 40), (9000, 50000)):
            want = X[rows, k:k + 40].astype(np.float64).T @ dY[rows, n:n + 40].astype(np.float64)
            _close(_host(dw[e, k:k + 40, n:n + 40]), want, 1.01, "dW")
    y = cf.grouped_gemm(_dev(X), dw, _i32(off))
    x = _dev(X)
    for e in (0, 2):
        rows = slice(int(off[e]), int(off[e + 1]))
        want = (x[rows].double() @ dw[e, :, -64:].double()).cpu().numpy()
        _close(_host(y[rows, -64:]), want, 1.01, "Y")


def test_wrapper_refusals():
    torch = torch_cuda()
    X = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(2, 64, 128, dtype=torch.bfloat16, device="cuda")
    off = _i32([0, 4, 8])
    for name, call in {
        "W": lambda: cf.grouped_gemm(X, W.half(), off),
        "W.*shape": lambda: cf.grouped_gemm(X, W[:, :32].contiguous(), off),
        "X is not contiguous": lambda: cf.grouped_gemm(X.T.contiguous().T, W, off),
        "W is not contiguous": lambda: cf.grouped_gemm(X, W.transpose(1, 2).contiguous().transpose(1, 2), off),
        "offsets.*dtype": lambda: cf.grouped_gemm(X, W, off.long()),
        "offsets.*shape": lambda: cf.grouped_gemm(X, W, off[:2]),
        "offsets is on cpu": lambda: cf.grouped_gemm(X, W, off.cpu()),
        "X has dtype": lambda: cf.grouped_gemm(X.float(), W, off),
        "out.*shape": lambda: cf.grouped_gemm(X, W, off, out=X),
        "preact": lambda: cf.grouped_gemm(X, W, off, preact=X),
        "unknown activation": lambda: cf.grouped_gemm(X, W, off, act="relu"),
        "dimensions": lambda: cf.grouped_gemm(X[0], W, off),
        "dY has shape": lambda: cf.grouped_gemm_wgrad(X, X[:4], off),
        "offsets is empty": lambda: cf.grouped_gemm_wgrad(X, X, off[:0]),
        "B has shape": lambda: cf.gemm_lora(X, W[0], None, W, W, off, off[:2]),
        "bias has dtype": lambda: cf.gemm_lora(X, W[0], X[0, :1].expand(128).contiguous(), W[:, :, :16].contiguous(),
                                               torch.zeros(2, 16, 128, dtype=X.dtype, device="cuda"), off, off[:2]),
    }.items():
        with pytest.raises(ValueError, match=name):
            call()
    with pytest.raises(cf.CfError, match="WORKSPACE_TOO_SMALL"):
        cf.grouped_gemm(X, W, off, workspace=cf.new_workspace(256))
    with pytest.raises(cf.CfError, match="UNSUPPORTED"):
        cf.grouped_gemm(X[:, :60].contiguous(), W[:, :60].contiguous(), off)
    with pytest.raises(cf.CfError, match="UNSUPPORTED"):
        cf.grouped_gemm(X, W, off, tuning=cf.tuning(n_slice=48))
    with pytest.raises(cf.CfError, match="UNSUPPORTED"):
        cf.grouped_gemm_wgrad(X, X, off, tuning=cf.tuning(n_slice=32))
    with pytest.raises(cf.CfError, match="INVALID_ARG"):
        cf.grouped_gemm(torch.zeros(8, 64, dtype=X.dtype, device="cuda"), W[:, :, :64].contiguous(), off,
                        out=(y := torch.zeros(8, 64, dtype=X.dtype, device="cuda")), preact=y)
    torch.cuda.synchronize()


@pytest.mark.parametrize("pair", [1, 2])
def test_a_wait_that_runs_out_is_reported(pair):
    """The accumulator-ready barrier waits for an arrival that nobody makes: every role drains, the call's status is
    CF_ERR_DEVICE_TIMEOUT, and the next call is right (on a workspace zeroed again)."""
    torch = torch_cuda()
    c = _layer(13)
    ws = cf.new_workspace(1 << 26)
    x, w1, off = _dev(c["x"]), _dev(c["w1"]), _i32(c["experts"])
    want = cf.grouped_gemm(x, w1, off)
    late = cf.tuning(extra_arrivals=1, timeout_us=2000, cluster_m=pair, n_slice=128)
    calls = [lambda t: cf.grouped_gemm(x, w1, off, workspace=ws, tuning=t),
             lambda t: cf.grouped_gemm_wgrad(x, want, off, workspace=ws, tuning=t),
             lambda t: cf.gemm_lora(x, _dev(c["wp"]), None, _dev(c["a"]), _dev(c["b"]), _i32(c["requests"]),
                                    _i32(c["adapters"]), workspace=ws, tuning=t)]
    for call in calls:
        call(late)
        assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
        cf.check(cf.cf_workspace_init(ws, ws.nbytes), "init")
        call(None)
        assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
    assert torch.equal(want, cf.grouped_gemm(x, w1, off, workspace=ws))
