"""Argument checks of the log probability calls: every refusal returns before
any CUDA call, so it is tested without a GPU."""
import pytest

from memory_fusion_gb300 import cf

P = 0x10000  # a 16-byte aligned address that no call below reads


@pytest.fixture(scope="module", autouse=True)
def built():
    from memory_fusion_gb300 import build
    build.build()


def _fwd(x=P, t=2 * P, lp=3 * P, lse=4 * P, h=5 * P, tl=6 * P, ti=7 * P, rows=4, v=100, stride=100, top=5, scale=1.0,
         dt=cf.CF_BF16, ws=8 * P, wsb=4096):
    return cf.cf_stitch_logprobs(x, t, lp, lse, h, tl, ti, rows, v, stride, top, scale, dt, ws, wsb, 0)


def _grad(x=P, t=2 * P, lse=3 * P, h=4 * P, dlp=5 * P, dlse=6 * P, dh=7 * P, dx=9 * P, rows=4, v=100, stride=100,
          dstride=100, scale=1.0, dt=cf.CF_BF16, ws=8 * P, wsb=4096):
    return cf.cf_stitch_logprobs_grad(x, t, lse, h, dlp, dlse, dh, dx, rows, v, stride, dstride, scale, dt, ws, wsb, 0)


@pytest.mark.parametrize("call", [_fwd, _grad])
def test_sizes(call):
    for kw in (dict(rows=-1), dict(v=-1), dict(stride=99), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(dt=3), dict(ws=None), dict(x=None)):
        assert call(**kw) == cf.CF_ERR_INVALID_ARG, kw
    big = dict(v=(1 << 24) + 1, stride=1 << 25)
    if call is _grad:
        big["dstride"] = 1 << 25
    for kw in (big, dict(rows=(1 << 27) + 1), dict(stride=(1 << 32) + 1)):
        assert call(**kw) == cf.CF_ERR_UNSUPPORTED, kw
    assert call(wsb=16) == cf.CF_ERR_WORKSPACE_TOO_SMALL
    assert call(rows=0, x=None) == cf.CF_OK
    assert call(x=P + 1) == cf.CF_ERR_MISALIGNED
    assert call(x=P + 2, dt=cf.CF_FP32) == cf.CF_ERR_MISALIGNED
    assert call(t=P + 4) == cf.CF_ERR_MISALIGNED


def test_forward():
    for kw in (dict(top=-1), dict(top=6, v=5), dict(t=None), dict(lp=None), dict(top=0), dict(tl=None, ti=None),
               dict(v=0, stride=0, top=0)):
        assert _fwd(**kw) == cf.CF_ERR_INVALID_ARG, kw
    assert _fwd(top=33) == cf.CF_ERR_UNSUPPORTED
    for n in ("lp", "lse", "h", "tl", "ti"):
        assert _fwd(**{n: P + 2}) == cf.CF_ERR_MISALIGNED, n


def test_gradient():
    for kw in (dict(lse=None), dict(dx=None), dict(t=None), dict(dlp=None), dict(h=None), dict(dh=None), dict(dstride=99),
               dict(t=None, dlp=None, dlse=None, h=None, dh=None), dict(dx=P, dstride=101)):
        assert _grad(**kw) == cf.CF_ERR_INVALID_ARG, kw
    assert _grad(v=0) == cf.CF_OK
    assert _grad(rows=1 << 27, v=1 << 20, stride=1 << 20, dstride=1 << 20) == cf.CF_ERR_UNSUPPORTED
    for n in ("lse", "h", "dlp", "dlse", "dh"):
        assert _grad(**{n: P + 2}) == cf.CF_ERR_MISALIGNED, n
    assert _grad(dx=P + 1) == cf.CF_ERR_MISALIGNED


def test_wrapper_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    for f in (lambda: cf.stitch_logprobs(x), lambda: cf.stitch_logprobs_grad(x, None, x[:, 0], dlse=x[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
