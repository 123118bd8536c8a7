"""Argument checks of the grouped GEMM and low-rank adapter calls: every
refusal returns before any CUDA call, so it is tested without a GPU."""
import pytest

from memory_fusion_gb300 import cf

P = 0x10000  # a 16-byte aligned address that no call below reads
WS = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from memory_fusion_gb300 import build
    build.build()


def _fwd(X=P, W=2 * P, off=3 * P, Y=4 * P, Z=None, T=8, N=64, K=64, E=2, dt=cf.CF_BF16, act=0, ws=5 * P, wsb=WS):
    return cf.cf_grouped_gemm(X, W, off, Y, Z, T, N, K, E, dt, act, ws, wsb, 0)


def _dgrad(dY=P, W=2 * P, off=3 * P, Z=None, dX=4 * P, T=8, N=64, K=64, E=2, dt=cf.CF_BF16, ws=5 * P, wsb=WS):
    return cf.cf_grouped_gemm_dgrad(dY, W, off, Z, dX, T, N, K, E, dt, ws, wsb, 0)


def _wgrad(X=P, dY=2 * P, off=3 * P, dW=4 * P, T=8, N=64, K=64, E=2, dt=cf.CF_BF16, ws=5 * P, wsb=WS):
    return cf.cf_grouped_gemm_wgrad(X, dY, off, dW, T, N, K, E, dt, ws, wsb, 0)


def _lora(X=P, W=2 * P, bias=None, A=6 * P, B=7 * P, off=3 * P, ad=8 * P, scale=None, Y=4 * P, T=8, N=64, K=64, S=2,
          L=3, R=16, dt=cf.CF_BF16, ws=5 * P, wsb=WS):
    return cf.cf_gemm_lora(X, W, bias, A, B, off, ad, scale, Y, T, N, K, S, L, R, dt, ws, wsb, 0)


CALLS = [_fwd, _dgrad, _wgrad, _lora]


@pytest.mark.parametrize("call", CALLS)
def test_sizes(call):
    groups = "S" if call is _lora else "E"
    for kw in (dict(T=-1), dict(N=0), dict(K=0), dict(N=-8), {groups: -1}, dict(dt=2), dict(dt=-1)):
        assert call(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for kw in (dict(N=65), dict(K=12), dict(N=1 << 25), dict(K=1 << 25), dict(T=1 << 31), {groups: 1025}):
        assert call(**kw) == cf.CF_ERR_UNSUPPORTED, kw


@pytest.mark.parametrize("call", CALLS)
def test_nothing_to_do(call):
    groups = "S" if call is _lora else "E"
    null = {"X": None, "dY": None, "off": None}
    kw = {k: v for k, v in null.items() if k in call.__code__.co_varnames}
    if call is not _wgrad:  # wgrad of no rows writes zeros
        assert call(T=0, **kw) == cf.CF_OK
    assert call(**{groups: 0}) == cf.CF_OK
    assert call(ws=None) == cf.CF_ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
def test_pointers(call):
    names = {"_fwd": ("X", "W", "off", "Y"), "_dgrad": ("dY", "W", "off", "dX"), "_wgrad": ("X", "dY", "off", "dW"),
             "_lora": ("X", "W", "A", "B", "off", "ad", "Y")}[call.__name__]
    for n in names:
        assert call(**{n: None}) == cf.CF_ERR_INVALID_ARG, n
        odd = 9 * P + (2 if n in ("off", "ad") else 8)
        assert call(**{n: odd}) == cf.CF_ERR_MISALIGNED, n
    assert call(ws=5 * P + 8) == cf.CF_ERR_MISALIGNED
    assert call(wsb=16) == cf.CF_ERR_WORKSPACE_TOO_SMALL


def test_aliases():
    assert _fwd(Y=P) == cf.CF_ERR_INVALID_ARG
    assert _fwd(Y=2 * P) == cf.CF_ERR_INVALID_ARG
    assert _fwd(Z=4 * P) == cf.CF_ERR_INVALID_ARG  # Z and Y are both written
    assert _fwd(Z=P) == cf.CF_ERR_INVALID_ARG
    assert _fwd(Z=9 * P + 4) == cf.CF_ERR_MISALIGNED
    assert _dgrad(dX=P) == cf.CF_ERR_INVALID_ARG
    assert _dgrad(Z=P) == cf.CF_ERR_INVALID_ARG
    assert _wgrad(dW=P) == cf.CF_ERR_INVALID_ARG
    assert _wgrad(dW=2 * P) == cf.CF_ERR_INVALID_ARG
    for y in (P, 2 * P, 6 * P, 7 * P):
        assert _lora(Y=y) == cf.CF_ERR_INVALID_ARG


def test_activation_and_rank():
    assert _fwd(act=2) == cf.CF_ERR_INVALID_ARG
    assert _lora(R=0) == cf.CF_ERR_INVALID_ARG
    assert _lora(L=-1) == cf.CF_ERR_INVALID_ARG
    for r in (4, 12, 136):
        assert _lora(R=r) == cf.CF_ERR_UNSUPPORTED
    assert _lora(bias=9 * P + 4) == cf.CF_ERR_MISALIGNED
    assert _lora(scale=9 * P + 2) == cf.CF_ERR_MISALIGNED


def test_wrapper_refusals():
    """The torch-level calls name the argument that does not fit."""
    torch = pytest.importorskip("torch")
    X, W, off = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16), \
        torch.zeros(3, dtype=torch.int32)
    for f in (lambda: cf.grouped_gemm(X, W, off), lambda: cf.grouped_gemm_dgrad(X, W, off),
              lambda: cf.grouped_gemm_wgrad(X, X, off),
              lambda: cf.gemm_lora(X, W[0], None, W, W, off, off[:2])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
