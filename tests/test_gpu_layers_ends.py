"""The norms around a block at the ends of what their calls allow: gradients of no
rows."""
import numpy as np
import pytest

from memory_fusion_gb300 import cf
from tests import test_gpu_block_norms as bn
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
