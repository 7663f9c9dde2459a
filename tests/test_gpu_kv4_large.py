"""Keys that a rotation takes past the largest 32-bit number: finite in 64 bits, so the cache in 4 bits
holds them as its largest values, not as NaN."""

import math

import pytest
import torch

import kv4_util as four
from test_gpu_kv4 import check_bytes, written


def bend(q, k, v):
    n, h, d = k.shape
    j = torch.arange(d)
    x = torch.ones(n, h, d)
    x[0::4] = 3.3e38 * (1 - 2 * (j % 2))
    x[1::4] = 2.5e38
    x[2::4, :, :d // 2] = 3.0e38
    x[3::4] = torch.where(j == 1, math.inf, 3.0e38)  # an infinity beside them is one still
    k.copy_(x.to(k.dtype).to(k.device))


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hk,d,tpp", [(2, 64, 3), (1, 128, 1), (3, 40, 2), (1, 256, 1)])
def test_keys_past_32_bits(hk, d, tpp, interleaved):
    n = 64
    cache, pool, slots, dev_slots, _, _, want, lay = written("bf16", hk, hk, d, tpp, n, rotary=d, interleaved=interleaved,
                                                             seed=d, bend=bend)
    far = want[0].abs()
    assert bool(((far >= 2.0 ** 128) & torch.isfinite(far)).any())
    check_bytes(cache, pool, slots, want, lay, tpp)
    k, v = (torch.zeros(n, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(k, v, *dev_slots)
    assert float(k[0].abs().max()) == 61440.0
    expect = four.values(*four.held(want[0]), d)
    assert torch.equal(k.cpu().double().nan_to_num(nan=7.0), expect.nan_to_num(nan=7.0))
    assert bool(torch.isnan(expect[3::4]).any()) and bool(torch.isfinite(expect[0::4]).all())
