"""The KV calls at the sizes they accept at most: 16384 requests, 2^30 cached tokens, positions
up to 2^31 - 1."""

import numpy as np
import pytest
import torch

import attn_exact as ax
import kv_util as ku
from test_gpu_attention_range import LOST as F16

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("append", [False, True])
def test_tables_of_16384_requests(append):
    from heterogeneous_lora_amd import runtime as rt
    rng = np.random.default_rng(1)
    n, tpp, width, planes = 16384, 2, 6, 2
    past, new = rng.integers(0, 6, n).astype(np.int32), rng.integers(0, 4, n).astype(np.int32)
    first = -(-past // tpp) if append else 0 * past
    n_ids = int((-(-(past + new) // tpp) - first).sum()) * planes
    n_pages = n_ids + 9
    pages = rng.permutation(n_pages)[:n_ids].astype(np.int32)
    old = rng.integers(0, n_pages, (planes, n, width)).astype(np.int32) if append else None
    want = ku.tables(past, new, pages, planes, tpp, width, n_pages, int(new.sum()), old)
    t = rt.KVTables(planes, n, width, int(new.sum()), table=None if old is None else torch.from_numpy(old).cuda())
    rt.KVCache(None, n_pages, tokens_per_page=tpp).tables(t, i32(pages), i32(past), i32(new), append=append)
    for k, x in want.items():
        assert np.array_equal(getattr(t, k).cpu().numpy(), x), k


def test_attention_of_16384_requests():
    lens = [i % 5 for i in range(16384)]
    lens[77], lens[16383] = 3000, 2000  # cut
    c = ax.dense_cache(lens, dtype="f16", hk=1, d=8, tpp=4, seed=3)
    q = torch.randn(16384, 2, 8, generator=torch.Generator().manual_seed(4)).half()
    cache, kt, vt = ax.to_gpu(c)
    some = [0, 1, 4, 76, 77, 78, 511, 512, 8191, 16382, 16383]
    ref = ax.attention(c, q[some], [(r, lens[r] - 1) for r in some], scale=0.3)
    for op in ("decode", "prefill"):
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        if op == "decode":
            cache.decode(q.cuda(), out, kt, vt, i32(lens), scale=0.3)
        else:
            cache.prefill(q.cuda(), out, kt, vt, i32(lens), torch.arange(16385, dtype=torch.int32, device="cuda"), scale=0.3)
        assert bool(out.isfinite().all())
        ku.check(out[some], ref.out, ax.bound(ref, "f16", *F16[op]), op)


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("window,prefix", [(1000, 0), (1, 0), (700, 300), (0, 0)])
def test_2_to_the_30_tokens(op, window, prefix):
    """A request as long as a table allows, its blocks on three pages of each kind: one for the
    first block, one for the last ones, one for all between."""
    d, tpp, blocks = 8, 1 << 18, 1 << 12
    n = (1 << 30) - 5
    g = torch.Generator().manual_seed(5)
    pages = torch.randn(6, tpp, d, generator=g).half()
    pages[5, :, 0] += 3
    table = lambda a: i32([[a] + [a + 1] * (blocks - 3) + [a + 2] * 2])
    from heterogeneous_lora_amd import runtime as rt
    cache = rt.KVCache(pages.cuda().view(-1), 6, page_elems=tpp * d, dtype="f16", n_kv_heads=1, head_dim=d, tokens_per_page=tpp)
    rows = 1 if op == "decode" else 3
    q = torch.randn(rows, 2, d, generator=g).half()
    out = torch.empty(rows, 2, d, dtype=torch.float16, device="cuda")
    opts = dict(scale=0.3, window=window, prefix_len=i32([prefix]) if prefix else None)
    if op == "decode":
        cache.decode(q.cuda(), out, table(0), table(3), i32([n]), **opts)
    else:
        cache.prefill(q.cuda(), out, table(0), table(3), i32([n]), i32([0, rows]), **opts)
    # the keys a row sees, page by page, with how often each place of a page is among them
    for i in range(rows):
        p = n - rows + i
        times = torch.zeros(3, tpp, dtype=torch.float64)
        if window:
            times[0, :prefix] = 1
            lo = p - window + 1
            assert lo // tpp >= blocks - 2
            for j in range(lo, p + 1):
                times[2, j % tpp] += 1
        else:
            times[0], times[1], times[2] = 1, blocks - 3, 1
            times[2, :p % tpp + 1] += 1
        w = times.view(-1) > 0
        k, v, many = pages[:3].view(-1, d)[w].double(), pages[3:].view(-1, d)[w].double(), times.view(-1)[w]
        for h in range(2):
            x = q[i, h].double()
            s = (k @ x) * 0.3
            e = torch.exp(s - s.max()) * many
            want, mass = e @ v / e.sum(), e @ v.abs() / e.sum()
            score = 2.0 ** -24 * (d + 16) * float((k.abs() @ x.abs()).max()) * 0.3 + 2.0 ** -22 * float(s.abs().max())
            # at most 2^17 values are added one after the other: a lane's share of a chunk
            sums = 2.0 ** -18 if window else 2.0 ** -7
            lost, floor = F16[op]
            floor = floor * float((v.abs() * many[:, None]).sum(0).max()) / float(e.sum()) if not window else floor * float(v.abs().sum(0).max())
            u, tiny = ku.half_step("f16")
            bound = (lost + 2 * score + sums) * mass + floor + u * want.abs() + tiny
            ku.check(out[i, h], want, bound, f"{op} row {i} head {h}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_to_2_to_the_31(interleaved):
    from heterogeneous_lora_amd import runtime as rt
    d, pos = 64, torch.tensor([0, 2 ** 24 + 1, 2 ** 30 - 1, 2 ** 31 - 1, 2 ** 31 - 2], dtype=torch.int32)
    q = torch.randn(5, 3, d, generator=torch.Generator().manual_seed(6)).half()
    rope = rt.Rope(d, interleaved=interleaved)
    pool = torch.zeros(1024, dtype=torch.float16, device="cuda")
    cache = rt.KVCache(pool, 8, page_elems=128, n_kv_heads=2, head_dim=64)
    out = torch.empty(5, 3, d, dtype=torch.float16, device="cuda")
    cache.write(q.cuda(), None, None, out, pos.cuda(), None, None, rope=rope)
    y, size = ku.written(q, pos, rope.turns_host, interleaved=interleaved, cos_sin_scale=1.0, norm=False, eps=0.0, weight=None)
    u, tiny = ku.half_step("f16")
    ku.check(out, y, u * y.abs() + 2.0 ** -20 * size + tiny, "far positions")
