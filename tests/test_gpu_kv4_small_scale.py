"""Attention over the cache in 4 bits with scales and rows of q so small that every score is next to
nothing: a row is the mean of the values it sees, and what it must not see stays unseen."""

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util

pytestmark = pytest.mark.gpu
SCALES = [1e-3, 1e-5, 1e-12, 1e-30]


def q_rows(n, hq, d, dtype, seed):
    """Ordinary rows, rows of zeros, rows of the type's smallest numbers."""
    q = torch.randn(n, hq, d, generator=torch.Generator().manual_seed(seed))
    q[0::3] = 0.0
    q[1::3] *= torch.finfo(util.TORCH[dtype]).smallest_normal
    return q.to(util.TORCH[dtype])


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hk,hq,d,past,new,cap", [(2, 4, 64, [0, 70], [33, 40], 0.0), (1, 128, 128, [40], [40], 0.0),
                                                  (1, 1, 200, [0], [50], 0.0), (1, 128, 64, [3], [40], 30.0)])
def test_prefill(hk, hq, d, past, new, cap, dtype, scale):
    lens = [a + b for a, b in zip(past, new)]
    c = four.Cache(np.random.default_rng(d), lens, dtype=dtype, hk=hk, d=d, tpp=3)
    q = q_rows(sum(new), hq, d, dtype, d)
    cache, kt, vt = c.to_gpu()
    out = torch.full_like(q, 7.0, device="cuda")
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets, scale=scale,
                  window=20, softcap=cap)
    rows = [(r, a + i) for r, (a, b) in enumerate(zip(past, new)) for i in range(b)]
    ref = four.attention(c, q, rows, scale=scale, window=20, cap=cap)
    back = sum(new) * hq // hk >= 4096 * len(lens)  # (keys read back first)
    util.check(out, ref.out, four.bound(ref, dtype, False, back=back), "prefill")


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("many", [False, True])
def test_decode(many, dtype, scale):
    lens = [1, 33, 100, 70, 300]
    c = four.Cache(np.random.default_rng(5), lens, dtype=dtype, hk=4, d=96, tpp=2,
                   blocks_more=2600000 // (4 * 2 * len(lens)) if many else 1)
    q = q_rows(len(lens), 8, 96, dtype, 6)
    cache, kt, vt = c.to_gpu()
    out = torch.full_like(q, 7.0, device="cuda")
    cache.decode(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale)
    ref = four.attention(c, q, [(r, n - 1) for r, n in enumerate(lens)], scale=scale)
    util.check(out, ref.out, four.bound(ref, dtype, True), "decode")
