"""The grouped GEMM and the low-rank adapters at the ends of their ranges: rows of a long request that share their last
tile with short ones, very long sums, the largest middle values, the activation's ends, sums that are exact.

Bounds are those of the other parity files (half a step of the 16-bit output plus the fp32 sums'), or equality where
every partial sum is a whole number that fp32 holds."""
import numpy as np
import pytest

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
