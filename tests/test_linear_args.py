"""Argument checks of the dense layer's calls: every refusal returns before
any CUDA call, so it is tested without a GPU."""
import pytest

from memory_fusion_gb300 import cf

P = 0x10000  # a 16-byte aligned address that no call below reads
WS = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from memory_fusion_gb300 import build
    build.build()


def _fwd(X=P, W=2 * P, b=None, R=None, Y=4 * P, Z=None, M=8, N=64, K=64, dt=cf.CF_BF16, act=0, ws=5 * P, wsb=WS):
    return cf.cf_gemm_linear(X, W, b, R, Y, Z, M, N, K, dt, act, ws, wsb, 0)


def _grad(dY=P, X=2 * P, W=3 * P, Z=None, dZ=None, dX=6 * P, dW=7 * P, db=8 * P, M=8, N=64, K=64, dt=cf.CF_BF16, act=0,
          ws=5 * P, wsb=WS):
    return cf.cf_gemm_linear_grad(dY, X, W, Z, dZ, dX, dW, db, M, N, K, dt, act, ws, wsb, 0)


@pytest.mark.parametrize("call", [_fwd, _grad])
def test_sizes(call):
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(N=-8), dict(dt=cf.CF_FP32), dict(dt=-1), dict(act=4),
               dict(act=-1), dict(ws=None)):
        assert call(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for kw in (dict(N=65), dict(K=12), dict(N=1 << 25), dict(K=1 << 25), dict(M=1 << 31), dict(N=1 << 24, K=1 << 15)):
        assert call(**kw) == cf.CF_ERR_UNSUPPORTED, kw
    assert call(wsb=16) == cf.CF_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=5 * P + 8) == cf.CF_ERR_MISALIGNED


def test_forward_pointers():
    assert _fwd(M=0, X=None, W=None, Y=None) == cf.CF_OK
    for n in ("X", "W", "Y"):
        assert _fwd(**{n: None}) == cf.CF_ERR_INVALID_ARG, n
    for n in ("X", "W", "Y", "b", "R", "Z"):
        assert _fwd(**{n: 9 * P + 8}) == cf.CF_ERR_MISALIGNED, n
    for kw in (dict(Y=P), dict(Y=2 * P), dict(Z=4 * P), dict(Z=P), dict(Z=2 * P), dict(R=9 * P, Z=9 * P)):
        assert _fwd(**kw) == cf.CF_ERR_INVALID_ARG, kw


def test_gradient_pointers():
    assert _grad(dY=None) == cf.CF_ERR_INVALID_ARG
    assert _grad(X=None) == cf.CF_ERR_INVALID_ARG
    assert _grad(W=None) == cf.CF_ERR_INVALID_ARG
    for kw in (dict(act=1), dict(act=1, Z=9 * P), dict(act=1, dZ=9 * P), dict(Z=9 * P), dict(dZ=9 * P)):
        assert _grad(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for n in ("dY", "X", "W", "dX", "dW", "db"):
        assert _grad(**{n: 9 * P + 8}) == cf.CF_ERR_MISALIGNED, n
    for kw in (dict(dX=P), dict(dX=2 * P), dict(dX=3 * P), dict(dW=P), dict(dW=2 * P), dict(dX=7 * P),
               dict(act=1, Z=9 * P, dZ=2 * P), dict(act=1, Z=9 * P, dZ=6 * P), dict(act=1, Z=6 * P, dZ=9 * P)):
        assert _grad(**kw) == cf.CF_ERR_INVALID_ARG, kw


def test_other_products_refuse_the_new_activations():
    for act in (cf.CF_ACT_SILU, cf.CF_ACT_RELU):
        assert cf.cf_grouped_gemm(P, 2 * P, 3 * P, 4 * P, None, 8, 64, 64, 1, cf.CF_BF16, act, 5 * P, WS,
                                  0) == cf.CF_ERR_INVALID_ARG
        assert cf.cf_gemm_fused_rownorm(P, 2 * P, None, 3 * P, 3 * P, 4 * P, 128, 512, 256, 1.0, 1e-5, act, 5 * P, WS,
                                        0) == cf.CF_ERR_INVALID_ARG


def test_wrapper_refusals():
    torch = pytest.importorskip("torch")
    X, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, 64, dtype=torch.bfloat16)
    for f in (lambda: cf.gemm_linear(X, W), lambda: cf.gemm_linear_grad(X, X, W)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
