"""The grouped GEMM and the low-rank adapters at the ends of their ranges: rows of a long request that share their last
tile with short ones, very long sums, the largest middle values, the activation's ends, sums that are exact.

Bounds are those of the other parity files (half a step of the 16-bit output plus the fp32 sums'), or equality where
every partial sum is a whole number that fp32 holds."""
import numpy as np
import pytest

from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import SENTINEL, _check, _host, _lora_case, _lora_run, _tuning
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
