"""The dense layer, the norms around a block and the log probabilities as a
program uses them: one after another forward and back, captured and replayed, on
other streams, from several threads, with workspaces in turn, without programmatic
launches, past 2^31 elements, over many gates, and with a wait that runs out."""
import threading

import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf
from tests import test_gpu_block_norms as bn
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def _model(dt, T=96, D=256, F=512, V=1000, seed=0):
    """Two layers with norms, gate and residual around them, a head and given tokens."""
    torch = torch_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0, kind=dt):
        return (torch.randn(*s, generator=g, device="cuda") * std + mean).to(kind)

    f32 = torch.float32
    return dict(h=normal(T, D, std=0.8), x=normal(T, D), gate=normal(4, D, std=0.3, mean=1.0),
                post=normal(D, std=0.1, mean=1.0, kind=f32), pre=normal(D, std=0.1, mean=1.0, kind=f32),
                w1=normal(D, F, std=D ** -0.5), b1=normal(F, std=0.1, kind=f32), w2=normal(F, D, std=F ** -0.5),
                b2=normal(D, std=0.1, kind=f32), last=normal(D, std=0.1, mean=1.0, kind=f32),
                head=normal(D, V, std=D ** -0.5), targets=torch.randint(0, V, (T,), generator=g, device="cuda"),
                dlp=normal(T, std=1 / T, mean=-1 / T, kind=f32), dh=normal(T, std=0.1 / T, kind=f32))


NORMS = dict(post="rms", pre="rms", scale=0.5, eps=1e-5)


def _run(m, kw=lambda: {}):
    """Log probabilities and every gradient of sum(dlp logprob + dh entropy); kw() makes each call's further arguments."""
    c = dict(post_weight=m["post"], pre_weight=m["pre"], gate=m["gate"], **NORMS)
    torch = torch_cuda()
    x1, y1 = cf.stitch_block_norms(m["h"], m["x"], **c, **kw())
    z = torch.empty(len(y1), m["w1"].shape[1], dtype=y1.dtype, device="cuda")
    a = cf.gemm_linear(y1, m["w1"], m["b1"], act="gelu_tanh", preact=z, **kw())
    x2 = cf.gemm_linear(a, m["w2"], m["b2"], residual=x1, **kw())
    x3, y3 = cf.stitch_block_norms(x2, None, pre="layer", pre_weight=m["last"], **kw())
    logits = cf.gemm_linear(y3, m["head"], **kw())
    lp, lse, ent, tl, ti = cf.stitch_logprobs(logits, m["targets"], top=5, **kw())
    dlogits = cf.stitch_logprobs_grad(logits, m["targets"], lse, m["dlp"], entropy=ent, dentropy=m["dh"], **kw())
    dy3, dhead, _ = cf.gemm_linear_grad(dlogits, y3, m["head"], bias=False, **kw())
    g3 = cf.stitch_block_norms_grad(dy3, None, x2, x3, pre="layer", pre_weight=m["last"], dx=False, **kw())
    da, dw2, db2 = cf.gemm_linear_grad(g3[0], a, m["w2"], **kw())
    dy1, dw1, db1 = cf.gemm_linear_grad(da, y1, m["w1"], act="gelu_tanh", preact=z, **kw())
    g1 = cf.stitch_block_norms_grad(dy1, g3[0], m["h"], x1, **c, **kw())
    return dict(lp=lp, ent=ent, ids=ti, top=tl, head=dhead, last=g3[5], w2=dw2, b2=db2, w1=dw1, b1=db1, h=g1[0], x=g1[1],
                gate=g1[2], post=g1[3], pre=g1[5])


def _exact(m):
    """The same in 64 bits, by automatic differentiation."""
    torch = torch_cuda()
    d = {k: v.double().requires_grad_() for k, v in m.items() if v.is_floating_point()}

    def rms(t, w):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-5) * w

    n = len(m["h"])
    x1 = d["x"] + 0.5 * d["gate"].repeat_interleave(n // 4, 0) * rms(d["h"], d["post"])
    z = rms(x1, d["pre"]) @ d["w1"] + d["b1"]
    x2 = torch.nn.functional.gelu(z, approximate="tanh") @ d["w2"] + d["b2"] + x1
    c = x2 - x2.mean(1, keepdim=True)
    logp = torch.log_softmax(rms(c, d["last"]) @ d["head"], 1)
    lp = logp[torch.arange(n), m["targets"]]
    ent = -(logp.exp() * logp).sum(1)
    (d["dlp"].detach() * lp + d["dh"].detach() * ent).sum().backward()
    return dict(lp=lp.detach(), ent=ent.detach(), **{k: d[k].grad for k in ("head", "last", "w2", "b2", "w1", "b1", "h", "x",
                                                                            "gate", "post", "pre")})


@pytest.mark.parametrize("name", ["bfloat16", "float16"])
def test_one_after_another(name):
    """Of each result the distance from the 64-bit one, as a whole (root of the sum of squares).  On the way to it lie at
    most 14 roundings to 16 bits, each off by at most half a step, eps / 2, of what it rounds, and gradients pass through
    products and norms whose sums keep that relative size (independent errors add as squares, far below the sum of 14
    that is allowed here)."""
    torch = torch_cuda()
    m = _model(getattr(torch, name))
    got, want = _run(m), _exact(m)
    bound = 14 * torch.finfo(getattr(torch, name)).eps / 2
    for k, w in want.items():
        err = (got[k].double() - w).norm() / w.norm()
        assert err < bound, (k, float(err), bound)


def test_captured_and_replayed():
    """Two graphs, each with workspaces of its own, replayed with other inputs, in turn; the results are the eager ones."""
    torch = torch_cuda()
    models = [_model(torch.bfloat16, seed=i) for i in range(2)]
    graphs = []
    for m in models:
        spaces = []

        def kw():
            spaces.append(cf.new_workspace(cf.cf_gemm_linear_workspace_size(96, 1000, 512)))
            return dict(workspace=spaces[-1])

        _run(m, kw)
        big = [cf.new_workspace(1 << 25) for _ in range(2)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _run(m, lambda: dict(workspace=big[0]))
        graphs.append((graph, out, big))
    for seed in (5, 6):
        for (graph, out, _), m in zip(graphs, models):
            for k, v in _model(torch.bfloat16, seed=seed).items():
                m[k].copy_(v)
            graph.replay()
        torch.cuda.synchronize()
        want = _run(_model(torch.bfloat16, seed=seed))
        for _, out, _ in graphs:
            for k in want:
                assert torch.equal(out[k], want[k]), k


def test_streams_and_threads():
    """The same bits from another stream, given or current, and from four threads at once."""
    torch = torch_cuda()
    m = _model(torch.bfloat16)
    want = _run(m)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given = _run(m, lambda: dict(stream=s))
    handle = _run(m, lambda: dict(stream=s.cuda_stream))
    with torch.cuda.stream(s):
        current = _run(m)
    torch.cuda.synchronize()
    got = [given, handle, current]

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = [_run(m) for _ in range(3)]
                torch.cuda.current_stream().synchronize()
            got.extend(out)
        except Exception as e:  # (an assertion in a thread would be lost)
            got.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 15
    for out in got:
        assert isinstance(out, dict), out
        for k in want:
            assert torch.equal(out[k], want[k]), k


def test_launches_without_overlap():
    torch = torch_cuda()
    m = _model(torch.float16)
    want, got = _run(m), _run(m, lambda: dict(tuning=cf.tuning(disable_pdl=1)))
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_one_workspace_in_turn():
    """Layer, its gradients, grouped products and adapters share one; the norms and log probabilities another."""
    torch = torch_cuda()
    ws = cf.new_workspace(1 << 25)
    m = _model(torch.bfloat16)
    off = torch.tensor([0, 40, 96], dtype=torch.int32, device="cuda")
    y = cf.gemm_linear(m["h"], m["w1"], workspace=ws)
    both = torch.stack([m["w1"], m["w1"]])
    for _ in range(3):
        assert torch.equal(cf.gemm_linear(m["h"], m["w1"], workspace=ws), y)
        g = cf.grouped_gemm(m["h"], both, off, workspace=ws)
        assert (g.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()
        cf.gemm_linear_grad(y, m["h"], m["w1"], workspace=ws)
    want = _run(m)
    got = _run(m, lambda: dict(workspace=ws))
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK


@pytest.mark.parametrize("shape,gates", [((5000, 512), (1, 10, 625, 1250, 2500)), ((20000, 40), (1, 8, 400, 10000)),
                                         ((4000, 333), (1, 5, 800, 2000)), ((2000, 1024), (2, 500, 2000)),
                                         ((1200, 9000), (1, 3, 400))], ids=str)
@pytest.mark.parametrize("norms,shift", [(("rms", "rms"), False), (("layer", "layer"), True)], ids=str)
def test_gates_across_stretches(shape, gates, norms, shift):
    """Stretches of several rows that begin and end inside a gate's rows, hold several gates, or lie inside one."""
    for n in gates:
        c, v, gate, kw = bn._case(shape, "bf16", *norms, n, shift)
        r = bn._rng(5)
        dy, dxo = bn._round(r.standard_normal(shape), "bf16"), bn._round(r.standard_normal(shape), "bf16")
        xo = bn._round(oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], "bf16")
        args = [bn._dev(a, "bf16") for a in (dy, dxo, c["h"], xo)]
        got = cf.stitch_block_norms_grad(*args, gate=bn._dev(gate, "bf16"), **{k: bn._dev(a) for k, a in v.items()}, **kw)
        ref = oracle.block_norms_grad(dy, dxo, c["h"], xo, gate=gate, **{k: a for k, a in v.items() if k != "pre_bias"}, **kw)
        bounds = bn._grad_bounds(dy, dxo, c, xo, v, gate, kw)
        for k, t in zip(bn.KEYS, got):
            if t is not None:
                bn._check(t, ref[k], bounds[k], "bf16" if k in ("h", "x", "gate") else "fp32", f"d{k} {n}")
        out, _ = cf.stitch_block_norms(args[2], bn._dev(c["x"], "bf16"), gate=bn._dev(gate, "bf16"),
                                       **{k: bn._dev(a) for k, a in v.items()}, **kw)
        bn._check(out, oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], bn._forward_bounds(c, v, gate, kw),
                  "bf16", f"x_out {n}")


def test_past_31_bits():
    """Rows behind the first 2^31 elements."""
    torch = torch_cuda()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("too little device memory")
    T, N = 530000, 4096
    rows = [0, 524287, 524288, 529999]
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(T, N, dtype=torch.bfloat16, device="cuda", generator=g)
    few = h[rows].clone()
    kw = dict(post="rms", pre="rms", eps=1e-5)
    want = cf.stitch_block_norms(few, few, **kw)
    xo, y = cf.stitch_block_norms(h, h, **kw)
    assert torch.equal(xo[rows], want[0]) and torch.equal(y[rows], want[1])
    dwant = cf.stitch_block_norms_grad(few, few, few, want[0], **kw)
    d = cf.stitch_block_norms_grad(h, h, h, xo, **kw, out=[y, None] + [None] * 5, dx=False)
    assert torch.equal(d[0][rows], dwant[0])
    del xo, y, d
    X, W = h[:, :64].contiguous(), torch.randn(64, 4096, dtype=torch.bfloat16, device="cuda", generator=g) / 8
    y = cf.gemm_linear(X, W, residual=h)
    assert torch.equal(y[rows], cf.gemm_linear(X[rows], W, residual=few))
    dx, dw, db = cf.gemm_linear_grad(y, X, W)
    assert torch.equal(dx[rows], cf.gemm_linear_grad(y[rows], X[rows], W, weight=False, bias=False)[0])
    total = sum(y[i:i + 10000].double().sum(0) for i in range(0, T, 10000))
    # fp32 sums of 530000 terms by chunks, warps and turns: about 900 + 8 + 608 additions each, 2^-24 of the sizes' sum
    size = sum(y[i:i + 10000].double().abs().sum(0) for i in range(0, T, 10000))
    assert ((db.double() - total).abs() <= 1600 * 2.0 ** -24 * size).all()


def test_wait_that_runs_out():
    """A row that never arrives: the status says so, the call ends, and the workspace serves again once it is zeroed."""
    torch = torch_cuda()
    h = torch.randn(700, 1024, device="cuda").bfloat16()
    ws = cf.new_workspace(cf.cf_stitch_block_norms_grad_workspace_size(700, 1024))
    kw = dict(post="rms", pre="rms", workspace=ws)
    want = cf.stitch_block_norms(h, h, **kw)
    t = cf.tuning(extra_arrivals=1, timeout_us=2000)
    cf.stitch_block_norms(h, h, tuning=t, **kw)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
    cf.stitch_block_norms_grad(h, h, h, h, tuning=t, **kw)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
    ws.zero_()
    got = cf.stitch_block_norms(h, h, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and cf.cf_get_device_status(ws)[0] == cf.CF_OK
    X, W = torch.randn(64, 256, device="cuda").bfloat16(), torch.randn(256, 512, device="cuda").bfloat16()
    ws = cf.new_workspace(cf.cf_gemm_linear_workspace_size(64, 512, 256))
    cf.gemm_linear(X, W, workspace=ws, tuning=t)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT


def test_depth_of_the_ring():
    """Two stages, or as many as fit: the same bits."""
    torch = torch_cuda()
    h = torch.randn(3000, 2048, device="cuda").bfloat16()
    want = cf.stitch_block_norms(h, h, post="layer", pre="rms")
    dwant = cf.stitch_block_norms_grad(h, h, h, want[0], post="rms", pre="rms")
    for n in (1, 2, 5, 20):
        t = cf.tuning(stages=n)
        got = cf.stitch_block_norms(h, h, post="layer", pre="rms", tuning=t)
        d = cf.stitch_block_norms_grad(h, h, h, want[0], post="rms", pre="rms", tuning=t)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(d[0], dwant[0])


@pytest.mark.parametrize("shape", [(700, 1024), (170, 8200), (320, 4095)], ids=str)
def test_depth_of_the_ring_with_means(shape):
    """A LayerNorm's means come with the row before where the ring holds two rows, and by themselves where it holds one;
    a row that never arrives ends both."""
    c, v, gate, kw = bn._case(shape, "bf16", "layer", "layer", 1, True)
    r = bn._rng(5)
    dy, dxo = (bn._round(r.standard_normal(shape), "bf16") for _ in range(2))
    xo = bn._round(oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], "bf16")
    args = [bn._dev(a, "bf16") for a in (dy, dxo, c["h"], xo)]
    dv, g = {k: bn._dev(a) for k, a in v.items()}, bn._dev(gate, "bf16")
    ref = oracle.block_norms_grad(dy, dxo, c["h"], xo, gate=gate, **{k: a for k, a in v.items() if k != "pre_bias"}, **kw)
    bounds = bn._grad_bounds(dy, dxo, c, xo, v, gate, kw)
    ws = cf.new_workspace(cf.cf_stitch_block_norms_grad_workspace_size(*shape))
    for n in (1, 2, 3, 8):
        got = cf.stitch_block_norms_grad(*args, gate=g, **dv, **kw, workspace=ws, tuning=cf.tuning(stages=n))
        assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
        for k, t in zip(bn.KEYS, got):
            bn._check(t, ref[k], bounds[k], "bf16" if k in ("h", "x", "gate") else "fp32", f"d{k} {n} stages")
    for n in (1, 2):
        t = cf.tuning(stages=n, extra_arrivals=1, timeout_us=2000)
        cf.stitch_block_norms_grad(*args, gate=g, **dv, **kw, workspace=ws, tuning=t)
        assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
        ws.zero_()
        cf.stitch_block_norms(args[2], args[3], gate=g, **dv, **kw, workspace=ws, tuning=t)
        assert cf.cf_get_device_status(ws)[0] == cf.CF_ERR_DEVICE_TIMEOUT
        ws.zero_()
    again = cf.stitch_block_norms_grad(*args, gate=g, **dv, **kw, workspace=ws)
    assert cf.cf_get_device_status(ws)[0] == cf.CF_OK
    bn._check(again[0], ref["h"], bounds["h"], "bf16", "dh")
