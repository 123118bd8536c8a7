"""Argument checks of the calls for the norms around a block: every refusal
returns before any CUDA call, so it is tested without a GPU."""
import pytest

from memory_fusion_gb300 import cf

P = 0x10000  # a 16-byte aligned address that no call below reads
WS = 1 << 40
NONE, RMS = cf.CF_NORM_NONE, cf.CF_NORM_RMS


@pytest.fixture(scope="module", autouse=True)
def built():
    from memory_fusion_gb300 import build
    build.build()


def _fwd(h=P, x=2 * P, gate=None, pw=None, pb=None, qw=None, qb=None, xo=3 * P, y=4 * P, rows=8, cols=64, gates=0,
         post=RMS, pre=RMS, dt=cf.CF_BF16, ws=5 * P, wsb=WS):
    return cf.cf_stitch_block_norms(h, x, gate, pw, pb, qw, qb, xo, y, rows, cols, gates, post, pre, 1.0, 1.0, 1e-5,
                                    dt, ws, wsb, 0)


def _grad(dy=P, dxo=2 * P, h=3 * P, xo=4 * P, gate=None, pw=None, pb=None, qw=None, dh=6 * P, dx=7 * P, dg=None,
          dpw=None, dpb=None, dqw=None, dqb=None, rows=8, cols=64, gates=0, post=RMS, pre=RMS, dt=cf.CF_BF16, ws=5 * P,
          wsb=WS):
    return cf.cf_stitch_block_norms_grad(dy, dxo, h, xo, gate, pw, pb, qw, dh, dx, dg, dpw, dpb, dqw, dqb, rows, cols,
                                         gates, post, pre, 1.0, 1.0, 1e-5, dt, ws, wsb, 0)


@pytest.mark.parametrize("call", [_fwd, _grad])
def test_sizes(call):
    for kw in (dict(rows=-1), dict(cols=-1), dict(gates=-1), dict(post=3), dict(pre=-1), dict(dt=3), dict(dt=-1),
               dict(gates=2), dict(gate=9 * P), dict(gate=9 * P, gates=3), dict(ws=None), dict(h=None)):
        assert call(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for kw in (dict(cols=32769), dict(rows=1 << 31)):
        assert call(**kw) == cf.CF_ERR_UNSUPPORTED, kw
    assert call(wsb=16) == cf.CF_ERR_WORKSPACE_TOO_SMALL
    assert call(h=P + 1) == cf.CF_ERR_MISALIGNED
    assert call(h=P + 2, dt=cf.CF_FP32) == cf.CF_ERR_MISALIGNED
    assert call(cols=0) == cf.CF_OK


def test_forward_pointers():
    assert _fwd(rows=0, h=None) == cf.CF_OK
    for kw in (dict(xo=None, y=None), dict(xo=4 * P), dict(post=NONE, pw=9 * P), dict(post=NONE, pb=9 * P),
               dict(pre=NONE), dict(pre=NONE, y=None, qw=9 * P), dict(gate=4 * P, gates=2), dict(gate=3 * P, gates=2)):
        assert _fwd(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for n in ("pw", "pb", "qw", "qb", "x", "xo", "y"):
        assert _fwd(**{n: 9 * P + 1}) == cf.CF_ERR_MISALIGNED, n


def test_gradient_pointers():
    for kw in (dict(dh=None), dict(dy=None, dxo=None), dict(xo=None), dict(post=NONE, pw=9 * P),
               dict(post=NONE, dpw=9 * P), dict(post=NONE, dpb=9 * P), dict(pre=NONE), dict(pre=NONE, dy=None, qw=9 * P),
               dict(dg=9 * P), dict(dy=None, dqw=9 * P), dict(dx=6 * P), dict(gate=9 * P, gates=2, dg=9 * P),
               dict(gate=6 * P, gates=2), dict(gate=9 * P, gates=2, dg=7 * P), dict(dpw=9 * P, dqw=9 * P)):
        assert _grad(**kw) == cf.CF_ERR_INVALID_ARG, kw
    for n in ("pw", "pb", "qw", "dpw", "dpb", "dqw", "dqb", "dy", "dxo", "xo", "dh", "dx", "ws"):
        assert _grad(**{n: 9 * P + 1}) == cf.CF_ERR_MISALIGNED, n


def test_other_calls_refuse_no_norm():
    assert cf.cf_gemm_fused_residual_norm(P, 2 * P, None, 3 * P, 4 * P, 4 * P, 6 * P, 128, 512, 256, 1.0, 1e-5, 0, NONE,
                                          5 * P, WS, 0) == cf.CF_ERR_INVALID_ARG


def test_wrapper_refusals():
    torch = pytest.importorskip("torch")
    h = torch.zeros(4, 64)
    for f in (lambda: cf.stitch_block_norms(h, h), lambda: cf.stitch_block_norms_grad(h, h, h, h, pre="rms")):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_gradient_of_no_rows_spares_the_gate():
    """It writes zeros to dgate, which is then no input either."""
    assert _grad(rows=0, gate=9 * P, gates=2, dg=9 * P) == cf.CF_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_fwd, _grad])
def test_a_gate_of_no_rows(call):
    """A gate goes with a number of gates, whatever the number of rows: nothing is divided by none."""
    for rows in (0, 8):
        assert call(rows=rows, gate=9 * P, gates=0) == cf.CF_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [_fwd, _grad])
def test_no_columns_with_gates(call):
    """A tensor of no columns has no address; the call has nothing to do."""
    assert call(cols=0, gate=None, gates=2) == cf.CF_OK
    assert call(cols=0, gate=9 * P, gates=2) == cf.CF_OK
    assert call(cols=0, gate=None, gates=3) == cf.CF_ERR_INVALID_ARG  # of 8 rows
