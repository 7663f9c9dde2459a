"""Attention where a request has more new tokens than cached ones (rows before position 0 see
the prefix alone), windows as wide as they can be, and offsets outside the rows."""

import numpy as np
import pytest
import torch

import kv_util as ku
from test_gpu_kv import _query

pytestmark = pytest.mark.gpu
MAX = 2 ** 31 - 1


def _run(c, q, new_offsets, **opts):
    cache, kt, vt = c.to_gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    prefix = opts.pop("prefix", None)
    cache.prefill(q.cuda(), out, kt, vt, i32(c.lens), i32(new_offsets), lse=lse,
                  prefix_len=None if prefix is None else i32(prefix), **opts)
    return out, lse.double().cpu()


@pytest.mark.parametrize("prefix", [None, [3, 0, 100]])
@pytest.mark.parametrize("window", [0, 1, 3, 89, 90, 91, 1 << 30, MAX])
def test_rows_before_the_first_key(window, prefix):
    lens, new = [5, 0, 90], [10, 4, 150]
    c = ku.Cache(np.random.default_rng(1), lens, dtype="f16", hk=2, d=64, tpp=3, blocks_more=0)
    assert c.max_blocks * 3 == 90
    rows = [(r, lens[r] - n + i) for r, n in enumerate(new) for i in range(n)]
    q = _query(c, 4, len(rows), "f16")
    want, bound, want_lse = ku.attention(c, q, rows, scale=0.1, window=window, prefix=prefix)
    out, lse = _run(c, q, [0, 10, 14, 164], scale=0.1, window=window, prefix=prefix)
    ku.check(out, want, bound, f"window {window}")
    assert torch.equal(torch.isinf(lse), torch.isinf(want_lse))
    f = torch.isfinite(want_lse)
    assert float((lse - want_lse).abs()[f].max()) < 1e-3


def test_offsets_outside_the_rows():
    lens = [40, 40, 40]
    c = ku.Cache(np.random.default_rng(2), lens, dtype="bf16", hk=1, d=64)
    q = _query(c, 2, 8, "bf16")
    rows = [(0, 35 + i) for i in range(5)] + [(2, 37 + i) for i in range(3)]
    want, bound, _ = ku.attention(c, q, rows, scale=0.1)
    out, _ = _run(c, q, [-3, 5, 5, 100], scale=0.1)  # rows 0..5, none, 5..8
    ku.check(out, want, bound, "clamped offsets")
    out, _ = _run(c, q, [5, 2, -7, 5], scale=0.1)    # decreasing: no row but the last request's
    ku.check(out[:5], *ku.attention(c, q[:5], [(2, 35 + i) for i in range(5)], scale=0.1)[:2], "decreasing offsets")
    assert (out[5:] == 7).all()
