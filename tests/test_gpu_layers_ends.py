"""The norms around a block and the log probabilities at the ends of what their
calls allow: gradients of no rows and of no columns, and of short rows, several of
which a worker takes in turn from its ring; entropy gradients so large that one
times a masked token's distance leaves fp32's range.

Bounds are those of the other parity files."""
import numpy as np
import pytest

import oracle
from memory_fusion_gb300 import cf
from tests import test_gpu_block_norms as bn
from tests import test_gpu_logprobs as lp
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gates", [1, 4])
def test_gradient_of_no_rows(gates, dt):
    """An empty batch: the gates' gradients are empty sums, as the weights' and biases' are."""
    torch = torch_cuda()
    e, g, w = (bn._dev(np.ones(s), t) for s, t in (((0, 64), dt), ((gates, 64), dt), ((64,), "fp32")))
    out = [None, None, torch.full_like(g, 7.0)] + [torch.full_like(w, 7.0) for _ in range(4)]
    v = dict(post_weight=w, post_bias=w, pre_weight=w, pre_bias=w)
    d = cf.stitch_block_norms_grad(e, e, e, e, post="rms", pre="layer", gate=g, **v, out=out)
    assert d[0].shape == d[1].shape == (0, 64)
    for want, got in zip(out[2:], d[2:]):
        assert got is want and not got.any()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_no_columns_with_gates(dt):
    torch = torch_cuda()
    n, g, w = (bn._dev(np.ones(s), t) for s, t in (((6, 0), dt), ((3, 0), dt), ((0,), "fp32")))
    kw = dict(post="rms", pre="rms", gate=g, post_weight=w, pre_weight=w)
    xo, y = cf.stitch_block_norms(n, n, **kw)
    assert xo.shape == y.shape == (6, 0)
    d = cf.stitch_block_norms_grad(n, n, n, xo, **kw)
    assert d[0].shape == (6, 0) and d[2].shape == (3, 0) and d[3].shape == d[5].shape == (0,)
    torch.cuda.synchronize()


# (workers of 152 SMs: 9728 for 37, 40 and 64 columns, 4864 for 128, 77824 for 1, 1216 for 333: 2 to 4 rows each)
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape,gates", [((20000, 40), (1, 400, 20000)), ((20000, 37), (8, 20000)), ((15000, 64), (0, 5)),
                                         ((12000, 128), (0, 12000)), ((80000, 1), (0, 2)), ((4000, 333), (5, 4000))], ids=str)
@pytest.mark.parametrize("norms,shift", [(("rms", "rms"), False), (("layer", "layer"), True)], ids=str)
def test_gradients_of_several_rows_a_worker(shape, gates, norms, shift, dt):
    """Every sum over the rows, which the groups of a CTA add in the place where their rings were."""
    torch = torch_cuda()
    ws = cf.new_workspace(cf.cf_stitch_block_norms_grad_workspace_size(*shape))
    for n in gates:
        c, v, gate, kw = bn._case(shape, dt, *norms, n, shift)
        r = bn._rng(5)
        dy, dxo = bn._round(r.standard_normal(shape), dt), bn._round(r.standard_normal(shape), dt)
        xo = bn._round(oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], dt)
        args = [bn._dev(a, dt) for a in (dy, dxo, c["h"], xo)]
        dv, g = {k: bn._dev(a) for k, a in v.items()}, bn._dev(gate, dt)
        got = cf.stitch_block_norms_grad(*args, gate=g, **dv, **kw, workspace=ws)
        ref = oracle.block_norms_grad(dy, dxo, c["h"], xo, gate=gate, **{k: a for k, a in v.items() if k != "pre_bias"}, **kw)
        bounds = bn._grad_bounds(dy, dxo, c, xo, v, gate, kw)
        for k, t in zip(bn.KEYS, got):
            assert (t is not None) == (k in ("h", "x") or k in v or (k == "gate" and n > 0)), k
            if t is not None:
                bn._check(t, ref[k], bounds[k], dt if k in ("h", "x", "gate") else "fp32", f"d{k} {n}")
        for _ in range(10):
            again = cf.stitch_block_norms_grad(*args, gate=g, **dv, **kw, workspace=ws)
            assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))
        out, _ = cf.stitch_block_norms(args[2], bn._dev(c["x"], dt), gate=g, **dv, **kw)
        bn._check(out, oracle.block_norms(c["h"], c["x"], gate=gate, **v, **kw)[0], bn._forward_bounds(c, v, gate, kw), dt,
                  f"x_out {n}")


@pytest.mark.parametrize("shape", [(24, 200), (6, 1111), (10, 4096)], ids=str)
def test_gradient_where_only_the_stream_was_used(shape):
    """y had no part in the loss: the call with pre "none", which reads neither x' nor Pre's weight, is the one of zeros
    for dy."""
    torch = torch_cuda()
    c, v, gate, kw = bn._case(shape, "bf16", "rms", "rms", 2, False)
    h, dxo, g, w = bn._dev(c["h"], "bf16"), bn._dev(c["x"], "bf16"), bn._dev(gate, "bf16"), bn._dev(v["post_weight"])
    kw = dict(kw, post_weight=w, gate=g)
    got = cf.stitch_block_norms_grad(None, dxo, h, None, **dict(kw, pre="none"))
    want = cf.stitch_block_norms_grad(torch.zeros_like(h), dxo, h, dxo, pre_weight=bn._dev(v["pre_weight"]), **kw)
    assert got[4:] == (None, None, None) and not want[5].any()
    for a, b in zip(got[:4], want[:4]):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="pre"):
        cf.stitch_block_norms_grad(None, dxo, h, None, **kw)


@pytest.mark.parametrize("N", [1, 8])
def test_most_rows(N):
    """The largest number of rows: workers without rows, or with fewer than others, write nothing behind the last one."""
    torch = torch_cuda()
    T, guard = 2 ** 31 - 512, 1 << 20
    if torch.cuda.mem_get_info()[0] < 4 * 2 * T * N + (8 << 30):
        pytest.skip("too little device memory")

    def rows():
        t = torch.full((T * N + guard,), 3.0, dtype=torch.bfloat16, device="cuda")
        return t, t[:T * N].view(T, N)

    def check(base, t, scale):
        assert (base[T * N:] == 3.0).all()
        for lo in range(0, T, 1 << 27):
            assert torch.equal(t[lo:lo + (1 << 27)], h[lo:lo + (1 << 27)] * scale)

    _, h = rows()
    h.view(-1)[:] = torch.randn(1 << 16, device="cuda").bfloat16().repeat(T * N // (1 << 16) + 1)[:T * N]
    base, out = rows()
    cf.stitch_block_norms(h, None, scale=2.0, out=out)
    check(base, out, 2.0)
    base.fill_(3.0)
    cf.stitch_block_norms(h, None, pre="rms", out=out, norm_out=(more := rows())[1])
    check(base, out, 1.0)
    x = h[-4096:].double()
    bound = bn.HALF["bf16"] + bn.K
    want = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5)
    assert (more[0][T * N:] == 3.0).all() and ((more[1][-4096:].double() - want).abs() <= bound * want.abs()).all()
    base.fill_(3.0)
    cf.stitch_block_norms_grad(None, h, h, None, scale=0.5, out=[out] + [None] * 6, dx=False)
    check(base, out, 0.5)


def test_dense_layer_of_most_rows():
    """The largest number of rows, whole numbers: equal to the call of its last rows, and nothing behind them."""
    torch = torch_cuda()
    M, tail, guard = 2 ** 31 - 512, 2000, 1 << 20
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("too little device memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    few = torch.randint(-2, 3, (1 << 16, 8), generator=g, device="cuda").bfloat16()
    W = torch.randint(-2, 3, (8, 8), generator=g, device="cuda").bfloat16()
    b = torch.randint(-2, 3, (8,), generator=g, device="cuda").float()
    X = torch.empty(M, 8, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 1 << 16):
        X[lo:lo + (1 << 16)] = few[:min(1 << 16, M - lo)]
    base = torch.full((M * 8 + guard,), 3.0, dtype=torch.bfloat16, device="cuda")
    Y = base[:M * 8].view(M, 8)
    cf.gemm_linear(X, W, b, act="relu", out=Y)
    want = cf.gemm_linear(few, W, b, act="relu")
    for lo in (0, M // (1 << 17) << 16, M >> 16 << 16):
        n = min(1 << 16, M - lo)
        assert torch.equal(Y[lo:lo + n], want[:n])
    assert (base[M * 8:] == 3.0).all()
    Y.zero_()
    Y[-tail:] = torch.randint(-2, 3, (tail, 8), generator=g, device="cuda").bfloat16()
    dx, dw, db = cf.gemm_linear_grad(Y, X, W)
    wx, ww, wb = cf.gemm_linear_grad(Y[-tail:].clone(), X[-tail:].clone(), W)
    assert torch.equal(dx[-tail:], wx) and not dx[:M - tail].any()
    assert torch.equal(dw, ww) and torch.equal(db, wb)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("scale,size", [(1.0, 2.0 ** 28), (1000.0, 64.0), (2.0 ** -10, 2.0 ** 40)], ids=str)
def test_large_entropy_gradients(scale, size, dt):
    """A masked token's probability is 0, and so is its gradient, whatever the loss is scaled by."""
    T, V = 9, 1003
    r = lp._rng(11)
    z = r.standard_normal((T, V)) * (2.5 / scale)
    mask = r.random((T, V)) < 0.5
    mask[0] = False
    mask[1, :] = np.arange(V) != 500
    t = r.integers(0, V, T)
    mask[np.arange(T), t] = False
    z[mask] = -np.inf
    z = lp._round(z, dt)
    zd, td = lp._dev(z, dt), lp._i64(t)
    f = cf.stitch_logprobs(zd, td, scale=scale)
    lse, ent = lp._host(f[1]), lp._host(f[2])
    dlp, dh = (size * r.standard_normal((2, T))).astype(np.float32)
    got = cf.stitch_logprobs_grad(zd, td, f[1], lp._dev(dlp), entropy=f[2], dentropy=lp._dev(dh), scale=scale)
    ref = oracle.logprobs_grad(z, t, dlogprob=dlp, dentropy=dh, scale=scale, lse=lse, entropy=ent)
    assert not lp._host(got)[mask].any()
    lp._within(got, ref, lp._grad_bound(z, t, scale, lse, ent, dlp, None, dh, dt, ref), f"{scale} {size}")


def test_log_probabilities_of_most_rows():
    torch = torch_cuda()
    T, V, n = 2 ** 27, 5, 1 << 14
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("too little device memory")
    few, t = lp._case((n, V, 0), "bf16", "masked")
    zf, tf = lp._dev(few, "bf16"), lp._i64(t)
    z, td = zf.repeat(T // n, 1), tf.repeat(T // n)
    got = cf.stitch_logprobs(z, td, top=2)
    want = cf.stitch_logprobs(zf, tf, top=2)
    lp._check(want, few, t, 1.0, 2)
    one = torch.ones(T, device="cuda")
    d = cf.stitch_logprobs_grad(z, td, got[1], one, entropy=got[2], dentropy=one)
    for lo in (0, T // 2, T - n):
        assert all(torch.equal(a[lo:lo + n], b) for a, b in zip(got, want))
    assert torch.equal(d[T - n:], cf.stitch_logprobs_grad(zf, tf, want[1], one[:n], entropy=want[2], dentropy=one[:n]))
    ref = oracle.logprobs_grad(few, t, dlogprob=np.ones(n), dentropy=np.ones(n), lse=lp._host(want[1]),
                               entropy=lp._host(want[2]))
    bound = lp._grad_bound(few, t, 1.0, lp._host(want[1]), lp._host(want[2]), np.ones(n), None, np.ones(n), "bf16", ref)
    lp._within(d[T - n:], ref, bound, "gradient")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_log_probabilities_of_the_largest_vocabulary(dt):
    z, t = lp._case((2, 2 ** 24, 0), dt, "masked")
    t = np.array([2 ** 24 - 1, 0])
    z[[0, 1], t] = 12.0
    got = cf.stitch_logprobs(lp._dev(z, dt), lp._i64(t), top=32)
    lp._check(got, z, t, 1.0, 32)
    d = cf.stitch_logprobs_grad(lp._dev(z, dt), lp._i64(t), got[1], lp._dev(np.ones(2)))
    ref = oracle.logprobs_grad(z, t, dlogprob=np.ones(2), lse=lp._host(got[1]))
    lp._within(d, ref, lp._grad_bound(z, t, 1.0, lp._host(got[1]), None, np.ones(2, np.float32), None, None, dt, ref), "gradient")
