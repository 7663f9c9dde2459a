"""One token over many keys in the cache in 4 bits, in spans of several rounds: tiles after tiles of a
wave, requests after requests of a workgroup, requests cut anywhere; with windows, the hole behind a
kept prefix, and what lies outside them no numbers. Against 64-bit references (kv4_shared)."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv4_shared as shared
import kv4_util as four
import kv_util as util
from heterogeneous_lora_amd import _lib

# dtype, KV heads, group, head_dim, tokens to a page, requests, longest; KV heads and runs of a wave, units
CASES = [
    ("f16", 8, 4, 128, 15, 64, 5000, (2, 2, 4)),
    ("bf16", 40, 1, 128, 3, 64, 1500, (10, 1, 4)),
    ("bf16", 4, 16, 64, 2, 130, 6000, (1, 4, 4)),
    ("f16", 8, 8, 256, 1, 100, 4000, (2, 2, 4)),
    ("bf16", 30, 1, 192, 1, 70, 1500, (7, 1, 4)),
    ("bf16", 4, 16, 224, 3, 130, 5000, (1, 2, 4)),
    ("f16", 2, 24, 96, 4, 260, 5000, (1, 4, 4)),
    ("f16", 1, 4, 128, 4, 600, 4500, (1, 4, 1)),
    ("bf16", 2, 8, 40, 7, 700, 2000, (1, 4, 2)),
    ("f16", 16, 1, 32, 8, 70, 3000, (4, 2, 4)),
    ("f16", 64, 1, 128, 1, 40, 2500, (16, 1, 4)),
    ("bf16", 56, 1, 96, 5, 60, 900, (14, 1, 4)),
    ("f16", 52, 1, 112, 2, 1100, 300, (13, 1, 4)),
    ("f16", 5, 3, 160, 2, 200, 3000, (2, 2, 4)),
    ("f16", 3, 3, 64, 6, 900, 1000, (1, 1, 4)),
]
# window, prefix, bias, cap
OPTIONS = [(0, 0, False, 0.0), (2500, 0, False, 0.0), (2500, 700, True, 0.0), (2200, 33, True, 30.0), (0, 0, True, 400.0)]


def lengths(rng, n, longest):
    """Short and long ones, none and one, next to multiples of rounds."""
    lens = [int(x) for x in rng.integers(longest // 3, longest + 1, n)]
    lens[::7] = [int(x) for x in rng.integers(0, 80, len(lens[::7]))]
    lens[:6] = [0, 1, longest, 64, 257, 128]
    return lens


def check(c, q, got, lse, **kw):
    ref = shared.attention(c, q, scale=c.d ** -0.5, **kw)
    worst = util.check(got, ref.out, four.bound(ref, c.dtype, True), "spans")
    fine = torch.isfinite(ref.lse)
    assert torch.equal(torch.isneginf(lse.cpu()), ~fine)
    assert float((lse.cpu().double() - ref.lse)[fine].abs().max()) <= float(2 * ref.d.max()) + 1e-5
    print(f"[margin] {worst:.3f}")


def case_of(dtype, hk, group, d, tpp, n, longest, option=OPTIONS[0], seed=0):
    window, prefix, bias, cap = option
    rng = np.random.default_rng(hk * d + n + seed)
    lens = lengths(rng, n, longest)
    need = -(-2500000 // (n * hk))  # (tables with room for that many keys are many)
    if window:
        window = max(window, need)
        lens = [x * 2 for x in lens]
    kept = rng.integers(0, prefix + 1, n) if prefix else None
    c = shared.Shared(hk + d, lens, dtype=dtype, hk=hk, d=d, tpp=tpp, max_len=max(max(lens), need, window + 1) + tpp, window=window,
                      prefix=kept)
    q = (torch.from_numpy(rng.standard_normal((n, hk * group, d))) * 1.5).to(util.TORCH[dtype])
    return c, q, dict(cap=cap, slopes=torch.linspace(0.0005, 0.02, hk * group) if bias else None)


def call(c, q, kw, ws=None, lens=None):
    cache, kt, vt = c.to_gpu()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.decode(q.cuda(), out, kt, vt, i32(c.lens if lens is None else lens), lse=lse, softcap=kw["cap"], window=c.window,
                 slopes=None if kw["slopes"] is None else kw["slopes"].cuda(),
                 prefix_len=None if c.prefix is None else i32([int(x) for x in c.prefix]), ws=ws)
    return out, lse


@pytest.mark.parametrize("case", CASES, ids=lambda x: "-".join(map(str, x[:7])))
def test_cases_are_in_several_rounds(case):
    c, q, _ = case_of(*case[:7])
    plan = shared.cut(c, q.shape[1])
    assert (plan.heads, plan.runs, plan.units) == case[7], plan
    assert plan.length >= 2 and plan.cut > 20, plan


@pytest.mark.gpu
@pytest.mark.timeout(120)
@pytest.mark.parametrize("case", CASES, ids=lambda x: "-".join(map(str, x[:7])))
def test_spans_of_several_rounds(case):
    c, q, kw = case_of(*case[:7])
    assert shared.cut(c, q.shape[1]).length >= 2
    got, lse = call(c, q, kw)
    check(c, q, got, lse, **kw)
    again, _ = call(c, q, kw)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.timeout(120)
@pytest.mark.parametrize("option", OPTIONS[1:], ids=str)
@pytest.mark.parametrize("case", [CASES[i] for i in (0, 1, 2, 5, 7, 9, 13)], ids=lambda x: "-".join(map(str, x[:7])))
def test_windows_and_kept_prefixes(case, option):
    c, q, kw = case_of(*case[:7], option=option)
    plan = shared.cut(c, q.shape[1])
    assert plan.spans and plan.length >= 2
    got, lse = call(c, q, kw)
    check(c, q, got, lse, **kw)


@pytest.mark.parametrize("window,prefix,cap", [(0, None, 0.0), (9, [3, 0, 40], 0.0), (5, None, 20.0)])
def test_the_reference(window, prefix, cap):
    """shared.attention beside kv4_util's over the same keys laid out one by one; and a key left out is seen."""
    lens = [40, 0, 23]
    c = shared.Shared(3, lens, dtype="f16", hk=2, d=40, tpp=3, max_len=45, pages=5, window=window, prefix=prefix)
    q = torch.randn(3, 6, 40, generator=torch.Generator().manual_seed(2)).half()
    slopes = torch.linspace(0.01, 0.1, 6)
    rows = [[torch.from_numpy(t[r].astype(np.int64))[torch.arange(n) // 3] * 3 + torch.arange(n) % 3 for t in (c.kt, c.vt)]
            for r, n in enumerate(lens)]
    dense = SimpleNamespace(hk=2, lens=lens, k=[c.x[k] for k, _ in rows], v=[c.x[v] for _, v in rows])
    want = four.attention(dense, q, [(r, n - 1) for r, n in enumerate(lens)], scale=0.3, cap=cap, window=window,
                          slopes=slopes, prefix=prefix)
    got = shared.attention(c, q, scale=0.3, cap=cap, slopes=slopes)
    for name in ("out", "mass", "total", "d", "lse"):
        a, b = getattr(got, name), getattr(want, name)
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-300), name
    c.lens[0] -= 1
    less = shared.attention(c, q, scale=0.3, cap=cap, slopes=slopes)
    assert bool(((less.out[0] - got.out[0]).abs() > four.bound(got, "f16", True)[0]).any())


@pytest.mark.gpu
@pytest.mark.timeout(120)
@pytest.mark.parametrize("option", [OPTIONS[0], OPTIONS[2]], ids=str)
@pytest.mark.parametrize("case", [CASES[i] for i in (0, 1, 3, 4, 9, 11)], ids=lambda x: "-".join(map(str, x[:7])))
def test_no_numbers_stay_with_their_head_and_request(case, option):
    """A step of V that is no number reaches its 32 dimensions of its head's rows, one of K its head's
    rows, a page outside the pool its request's: bit for bit the rest is as without them."""
    c, q, kw = case_of(*case[:7], option=option)
    g, sb, size = four.layout(c.hk, c.d)
    group, tpp = q.shape[1] // c.hk, c.tpp
    kt, vt = c.kt.copy(), c.vt.copy()
    clean, clean_lse = call(c, q, kw)
    long = [r for r, n in enumerate(c.lens) if n > 600]
    head, last = c.hk - 2 if c.hk > 2 else 0, g - 1
    for page, table, other, r in ((c.n_pages - 2, c.vt, vt, long[3]), (c.n_pages - 1, c.kt, kt, long[9])):
        j = int(c.seen(r)[len(c.seen(r)) // 2])
        c.pool[page] = c.pool[int(other[r, j // tpp])]
        c.pool[page, (j % tpp) * size + c.hk * 16 * g + head * sb + last] = 255
        table[r, j // tpp] = page
    c.kt[long[12], int(c.seen(long[12])[5]) // tpp] = c.n_pages
    c.vt[long[15], (c.lens[long[15]] - 1) // tpp] = -1
    got, lse = call(c, q, kw)
    rows = slice(head * group, (head + 1) * group)
    bad, bad_lse = torch.zeros(got.shape, dtype=torch.bool), torch.zeros(lse.shape, dtype=torch.bool)
    bad[long[3], rows, 32 * last:] = True
    bad[long[9], rows] = bad_lse[long[9], rows] = True
    bad[long[12]] = bad_lse[long[12]] = True
    bad[long[15]] = True
    got, lse, clean, clean_lse = got.cpu(), lse.cpu(), clean.cpu(), clean_lse.cpu()
    assert torch.equal(torch.isnan(got), bad) and torch.equal(torch.isnan(lse), bad_lse)
    assert torch.equal(got[~bad], clean[~bad]) and torch.equal(lse[~bad_lse], clean_lse[~bad_lse])


@pytest.mark.gpu
@pytest.mark.timeout(120)
def test_replays_with_other_lengths():
    """A captured call, replayed while the lengths change, between eager calls in the same workspace."""
    c, q, kw = case_of(*CASES[1][:7])
    cache, kt, vt = c.to_gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seq, out = i32(c.lens), torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    need = cache.workspace_size(cache._kv(len(c.lens), c.max_blocks), _lib.Attn(n_q_heads=q.shape[1]), 0)
    ws, qd = torch.zeros(need, dtype=torch.uint8, device="cuda"), q.cuda()
    bound = cache.bind_decode(qd, out, kt, vt, seq, ws=ws)
    bound()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.bind_decode(qd, out, kt, vt, seq, ws=ws)()
    rng = np.random.default_rng(8)
    for turn in range(4):
        lens = [int(x) for x in rng.permutation(c.lens)] if turn % 2 else [min(n, 90 + turn) for n in c.lens]
        lens = [min(a, b) for a, b in zip(lens, c.lens)]  # (tables end at a request's own length)
        seq.copy_(i32(lens))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        out.fill_(7.0)
        bound()
        assert torch.equal(replayed.view(torch.int16), out.view(torch.int16))
        c.lens = lens
        ref = shared.attention(c, q, scale=c.d ** -0.5)
        util.check(replayed, ref.out, four.bound(ref, c.dtype, True), f"replay {turn}")
