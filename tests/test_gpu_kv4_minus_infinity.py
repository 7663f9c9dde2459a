"""One token over the cache in 4 bits whose scores are all minus infinity (bf16 q times K past the
largest 32-bit number): 0 with lse minus infinity, whatever V holds, also where a request is cut; and
scores of which only some are."""

import math

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("hk,hq,d,n", [(4, 4, 64, 20), (4, 8, 128, 700), (1, 16, 256, 300), (8, 8, 96, 1500)])
def test_all_scores(hk, hq, d, n, many):
    lens = [n, 40]
    c = four.Cache(np.random.default_rng(d), lens, dtype="bf16", hk=hk, d=d, tpp=4,
                   blocks_more=2600000 // (hk * 2 * 4) if many else 1)
    k = torch.zeros(n, hk, d, dtype=torch.float64)
    k[..., 0] = -6000.0
    c.put(0, slice(0, n), 0, k)
    nan = torch.full((1, hk, d), math.nan, dtype=torch.float64)
    c.put(0, slice(3, 4), 1, nan)
    c.put(0, slice(n - 2, n - 1), 1, nan)
    q = torch.randn(2, hq, d, generator=torch.Generator().manual_seed(1))
    q[0] = 0.0
    q[0, :, 0] = 3e38
    q = q.to(torch.bfloat16)
    cache, kt, vt = c.to_gpu()
    out = torch.full_like(q, 7.0, device="cuda")
    lse = torch.zeros(2, hq, device="cuda")
    cache.decode(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse)
    assert bool((out[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    ref = four.attention(c, q[1:], [(1, 39)], scale=d ** -0.5)
    util.check(out[1:], ref.out, four.bound(ref, "bf16", True), "the other request")
    # one key with a score of 0: the row is its V, and what the others hold is no number
    c.put(0, slice(1, 2), 0, torch.zeros(1, hk, d, dtype=torch.float64))
    for bad in (True, False):
        if not bad:
            for j in (3, n - 2):
                c.put(0, slice(j, j + 1), 1, torch.ones(1, hk, d, dtype=torch.float64))
        cache, kt, vt = c.to_gpu()
        cache.decode(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse)
        if bad:
            assert bool(torch.isnan(out[0]).all())
        else:
            assert torch.equal(out[0].cpu(), c.v[0][1].repeat_interleave(hq // hk, 0))
        assert bool((lse[0] == 0).all())
