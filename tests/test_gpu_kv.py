"""KV cache and attention operators on the GPU against plain 64-bit references (kv_util):
types, head layouts, lengths from zero up, tables, masks, strides, bad device data,
infinities and NaN in masked places, streams and graph replays."""

import numpy as np
import pytest
import torch

import kv_util as ku

pytestmark = pytest.mark.gpu
T = ku.TORCH


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from heterogeneous_lora_amd import _lib, runtime
    _lib.load()
    return runtime


# ---------------------------------------------------------------- tables

TABLES = {
    "one token": dict(past=[0], new=[1], planes=2, tpp=1),
    "no request": dict(past=[], new=[], planes=2, tpp=1, spare=3),
    "nothing new": dict(past=[5, 0, 7], new=[0, 0, 0], planes=4, tpp=2, spare=2),
    "ragged": dict(past=[0, 3, 64, 65, 0, 130], new=[7, 1, 0, 64, 0, 129], planes=6, tpp=1, width=300),
    "pages end inside": dict(past=[1, 5, 8, 0, 15], new=[6, 1, 1, 3, 2], planes=2, tpp=5),
    "many planes": dict(past=[3, 70], new=[1, 2], planes=131, tpp=3, width=90),
    "odd planes": dict(past=[400, 1500], new=[10, 7], planes=3, tpp=1, width=2000),
    "many requests": dict(past=[i % 7 for i in range(700)], new=[(i * 5) % 3 for i in range(700)], planes=2, tpp=2),
    "padded step": dict(past=[9, 2], new=[1, 1], planes=2, tpp=4, spare=700),
    "too many tokens": dict(past=[4, 4, 4], new=[300, 300, 300], planes=2, tpp=1, spare=-350),
    "past the table": dict(past=[10, 0], new=[40, 3], planes=2, tpp=2, width=17),
    "short list": dict(past=[10, 10], new=[5, 5], planes=2, tpp=1, drop=9),
    "negative lengths": dict(past=[-3, 4, -2147483648], new=[2, -5, 1], planes=2, tpp=2),
    "pages outside": dict(past=[3, 4], new=[2, 6], planes=2, tpp=2, bad=True),
}


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("name", sorted(TABLES))
def test_tables(rt, name, append):
    c = dict(TABLES[name])
    rng = np.random.default_rng(1)
    past, new, planes, tpp = c["past"], c["new"], c["planes"], c["tpp"]
    p, w = [max(x, 0) for x in past], [max(x, 0) for x in new]
    first = [-(-a // tpp) if append else 0 for a in p]
    blocks = [-(-(a + b) // tpp) for a, b in zip(p, w)]
    width = c.get("width", max(blocks + [0]) + 3)
    n_ids = sum(b - f for b, f in zip(blocks, first)) * planes
    n_pages = n_ids + 50
    pages = rng.permutation(n_pages)[:n_ids].astype(np.int32)
    if c.get("bad"):
        pages[::3] = [-1, -2147483648, n_pages, 2147483647][:1] * len(pages[::3])
        pages[1::5] = n_pages
    pages = pages[:max(n_ids - c.get("drop", 0), 0)]
    n_tok = max(sum(w) + c.get("spare", 0), 0)
    old = rng.integers(0, n_pages, (planes, len(p), width)).astype(np.int32) if append else None
    want = ku.tables(past, new, pages, planes, tpp, width, n_pages, n_tok, old)
    t = rt.KVTables(planes, len(p), width, n_tok, table=None if old is None else torch.from_numpy(old).cuda())
    cache = rt.KVCache(None, n_pages, tokens_per_page=tpp)
    to = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.tables(t, torch.from_numpy(pages).cuda(), to(past), to(new), append=append)
    for k, x in want.items():
        got = getattr(t, k).cpu().numpy()
        assert np.array_equal(got, x), (k, np.argwhere(got != x)[:5])


def test_tables_length_past_int32(rt):
    """Lengths whose sum passes 2^31, and more blocks than any table: nothing out of range."""
    t = rt.KVTables(2, 2, 4, 8)
    cache = rt.KVCache(None, 16)
    big = torch.tensor([2147483647, 2147483647], dtype=torch.int32, device="cuda")
    cache.tables(t, torch.arange(16, dtype=torch.int32, device="cuda"), big, big)
    assert t.seq_len.tolist() == [2147483647] * 2 and t.q_offsets.tolist() == [0, 8, 8]
    assert t.token_request.tolist() == [0] * 8 and t.position[0].item() == 2147483647
    assert (t.slots == -1).all()
    assert t.table[0, 0].tolist() == [0, 2, 4, 6] and t.table[1, 0].tolist() == [1, 3, 5, 7]
    assert (t.table[:, 1] == -1).all()


# ---------------------------------------------------------------- write

WRITE = {
    "one token": dict(t=1, hq=4, hk=4, d=64, rot=64),
    "half of the head": dict(t=5, hq=6, hk=2, d=128, rot=64, norm=True),
    "halves of 36": dict(t=7, hq=4, hk=2, d=72, rot=72, norm=True),
    "halves of 12": dict(t=3, hq=2, hk=1, d=96, rot=24),
    "small head": dict(t=9, hq=3, hk=3, d=8, rot=8, norm=True),
    "no rotation": dict(t=4, hq=4, hk=4, d=80, rot=0, norm=True, weight=False),
    "widest head": dict(t=6, hq=8, hk=1, d=256, rot=256, norm=True),
    "odd pieces": dict(t=4, hq=5, hk=5, d=40, rot=16, norm=True),
    "many tokens": dict(t=4500, hq=2, hk=1, d=64, rot=64, tpp=3),
    "many heads": dict(t=2, hq=64, hk=8, d=128, rot=128, tpp=2, norm=True),
}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("name", sorted(WRITE))
def test_write(rt, name, interleaved, dtype):
    c = WRITE[name]
    t, hq, hk, d, rot, tpp = c["t"], c["hq"], c["hk"], c["d"], c["rot"], c.get("tpp", 1)
    norm = c.get("norm", False)
    rng = np.random.default_rng(2)
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(t, (hq + 2 * hk) * d + 8, generator=g).to(T[dtype])
    cut = lambda x: [y.unflatten(1, (-1, d)) for y in (x[:, :hq * d], x[:, hq * d:(hq + hk) * d],
                                                       x[:, (hq + hk) * d:(hq + 2 * hk) * d])]
    q, k, v = cut(packed)
    P = tpp * hk * d + 8
    n_pages = 2 * (-(-t // tpp)) + 3
    pool = torch.randn(n_pages, P, generator=g).to(T[dtype])
    order = rng.permutation(n_pages)
    place = lambda i: order[i * (-(-t // tpp)) + np.arange(t) // tpp] * tpp + np.arange(t) % tpp
    ks, vs = place(0).astype(np.int64), place(1).astype(np.int64)
    pos = rng.integers(0, 1_000_000, t).astype(np.int32)
    if t > 3:  # a padding token, and slots outside the pool
        pos[1] = -1
        ks[2], vs[0], vs[2] = -1, n_pages * tpp, (1 << 40)
    kw = kq = None
    if norm and c.get("weight", True):
        kq, kw = [(1 + 0.3 * torch.randn(d, generator=g)).to(T[dtype]) for _ in range(2)]
    cs = 1.25
    rope = rt.Rope(rot, interleaved=interleaved, cos_sin_scale=cs) if rot else None
    turns = torch.from_numpy(rope.turns_host) if rot else torch.zeros(0, dtype=torch.float64)
    cache = rt.KVCache(pool.cuda(), n_pages, page_elems=P, dtype=dtype, n_kv_heads=hk, head_dim=d, tokens_per_page=tpp)
    gq, gk, gv = cut(packed.cuda())
    out = torch.full((t, hq + 1, d), 7.0, dtype=T[dtype], device="cuda")[:, :hq]
    dev = lambda x: None if x is None else (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()
    args = (gq, gk, gv, out, dev(pos), dev(ks), dev(vs))
    kwargs = dict(rope=rope, norm=norm, q_weight=dev(kq), k_weight=dev(kw), eps=1e-5)
    cache.write(*args, **kwargs)
    live = torch.from_numpy(pos >= 0)
    u, tiny = ku.half_step(dtype)
    opts = dict(interleaved=interleaved, cos_sin_scale=cs, norm=norm, eps=1e-5)
    yq, sq = ku.written(q, torch.from_numpy(pos), turns, weight=kq, **opts)
    yq[~live] = 7.0
    ku.check(out.cpu(), yq, u * yq.abs() + 2.0 ** -20 * sq + tiny, f"{name} q")
    yk, sk = ku.written(k, torch.from_numpy(pos), turns, weight=kw, **opts)
    want, bound = pool.double(), torch.zeros(n_pages, P, dtype=torch.float64) + 1e-300
    for i in range(t):
        for y, s, slot in ((yk, 2.0 ** -20 * sk + u * yk.abs() + tiny, int(ks[i])),
                           (v.double(), torch.zeros_like(yk) + 1e-300, int(vs[i]))):
            if pos[i] >= 0 and 0 <= slot // tpp < n_pages:
                o = slot % tpp * hk * d
                want[slot // tpp, o:o + hk * d] = y[i].reshape(-1)
                bound[slot // tpp, o:o + hk * d] = s[i].reshape(-1)
    ku.check(cache.pool.cpu(), want, bound, f"{name} pool")
    # q alone, in place: the same bits
    cache.write(gq, None, None, gq, dev(pos), None, None, **kwargs)
    assert torch.equal(gq[live.cuda()], out[live.cuda()])


# ---------------------------------------------------------------- attention

ODD_LENS = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]
DECODE = {
    "lengths": dict(lens=ODD_LENS, hk=2, group=1, d=64),
    "pages end inside": dict(lens=ODD_LENS, hk=2, group=2, d=128, tpp=5, slack=8),
    "heads of 8": dict(lens=[0, 5, 70], hk=1, group=3, d=8, tpp=2),
    "heads of 40": dict(lens=[1, 40], hk=2, group=1, d=40),
    "heads of 72": dict(lens=[1, 40, 129], hk=2, group=2, d=72),
    "heads of 80": dict(lens=[1, 40, 129], hk=2, group=2, d=80, tpp=3),
    "heads of 96": dict(lens=[1, 40, 129], hk=1, group=8, d=96),
    "heads of 120": dict(lens=[64, 3], hk=1, group=4, d=120),
    "heads of 160": dict(lens=[7, 131], hk=2, group=4, d=160),
    "heads of 192": dict(lens=[7, 131], hk=1, group=1, d=192),
    "heads of 256": dict(lens=[0, 7, 131], hk=1, group=16, d=256, tpp=2),
    "17 to a key head": dict(lens=[5, 100], hk=2, group=17, d=64),
    "many requests": dict(lens=[(i * 7) % 50 for i in range(150)], hk=1, group=1, d=64, tpp=4),
    "one long": dict(lens=[3000], hk=1, group=2, d=64, tpp=2),
    "long and short": dict(lens=[1, 2500, 0, 131, 700], hk=2, group=1, d=128),
    "window": dict(lens=[0, 1, 30, 64, 200, 900], hk=2, group=2, d=64, window=64),
    "window and prefix": dict(lens=[0, 1, 30, 64, 200, 900], hk=1, group=2, d=128, window=33, prefix=[4, 4, 50, 1, 7, 131], tpp=3),
    "window of one": dict(lens=[1, 2, 77], hk=1, group=1, d=64, window=1),
    "cap": dict(lens=[1, 33, 200], hk=2, group=2, d=64, cap=5.0, k_scale=3.0),
    "slopes": dict(lens=[1, 33, 200], hk=2, group=2, d=64, slopes=True),
    "everything": dict(lens=[1, 33, 700], hk=2, group=4, d=96, tpp=4, cap=20.0, slopes=True, window=100, prefix=[3, -5, 9]),
}


def _query(c, hq, n, dtype, seed=5):
    return (torch.randn(n, hq, c.d, generator=torch.Generator().manual_seed(seed)) * 1.5).to(T[dtype])


def _attn(rt, name, spec, dtype, new=None):
    rng = np.random.default_rng(4)
    opts = {k: spec[k] for k in ("hk", "d", "tpp", "slack", "k_scale") if k in spec}
    c = ku.Cache(rng, spec["lens"], dtype=dtype, **opts)
    hq = c.hk * spec["group"]
    slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq) if spec.get("slopes") else None
    prefix = spec.get("prefix")
    rows = [(r, n - 1) for r, n in enumerate(c.lens)] if new is None else \
        [(r, c.lens[r] - w + i) for r, w in enumerate(new) for i in range(w)]
    q = _query(c, hq, len(rows), dtype)
    ref = dict(scale=0.3 * c.d ** -0.25, cap=spec.get("cap", 0.0), window=spec.get("window", 0))
    out = torch.full((len(rows), hq + 1, c.d), 7.0, dtype=T[dtype], device="cuda")[:, :hq]
    lse = torch.full((len(rows), hq), 7.0, device="cuda")
    dev = dict(scale=ref["scale"], softcap=ref["cap"], window=ref["window"], lse=lse,
               slopes=None if slopes is None else slopes.cuda(),
               prefix_len=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"))
    seq = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    return c, q, rows, dict(ref, slopes=slopes, prefix=prefix), out, lse, dev, seq


def _check_attn(what, c, q, rows, ref, out, lse):
    want, bound, want_lse = ku.attention(c, q, rows, **ref)
    worst = ku.check(out, want, bound, what)
    got = lse.double().cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(want_lse)), what
    f = torch.isfinite(want_lse)
    # scores within the bound's error, sums in 32 bits
    assert float((got - want_lse).abs()[f].max() if f.any() else 0.0) < 1e-3, what
    print(f"[margin] {what}: {worst:.3f} of the bound", flush=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode(rt, name, dtype):
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, name, DECODE[name], dtype)
    cache, kt, vt = c.to_gpu()
    cache.decode(q.cuda(), out, kt, vt, seq, **dev)
    _check_attn(f"decode {name} {dtype}", c, q, rows, ref, out, lse)


PREFILL = {
    "prompts": dict(lens=[1, 17, 64, 130, 0, 5], new=[1, 17, 64, 130, 0, 5], hk=2, group=1, d=64),
    "continued": dict(lens=[100, 129, 200, 64], new=[1, 65, 0, 3], hk=2, group=2, d=128, tpp=3),
    "row tiles": dict(lens=[300, 40], new=[290, 40], hk=1, group=3, d=64, tpp=2),
    "heads of 8": dict(lens=[5, 70], new=[5, 20], hk=1, group=3, d=8, tpp=2),
    "heads of 72": dict(lens=[40, 99], new=[40, 9], hk=1, group=2, d=72),
    "heads of 96": dict(lens=[40, 99], new=[40, 9], hk=2, group=1, d=96, tpp=5, slack=16),
    "heads of 120": dict(lens=[40], new=[33], hk=1, group=1, d=120),
    "heads of 160": dict(lens=[40, 99], new=[40, 9], hk=1, group=4, d=160),
    "heads of 256": dict(lens=[40, 99], new=[40, 70], hk=1, group=2, d=256, tpp=2),
    "shared by 17": dict(lens=[50], new=[20], hk=1, group=17, d=64),
    "window": dict(lens=[1, 150, 260], new=[1, 150, 60], hk=1, group=2, d=64, window=33),
    "window of one": dict(lens=[70, 140], new=[70, 2], hk=1, group=1, d=64, window=1),
    "prefix": dict(lens=[100, 140, 30], new=[100, 70, 30], hk=1, group=2, d=64, prefix=[64, 100, 200]),
    "window and prefix": dict(lens=[100, 300, 30], new=[100, 70, 30], hk=1, group=2, d=128, window=20, prefix=[5, 150, -1]),
    "cap": dict(lens=[100, 30], new=[60, 30], hk=2, group=1, d=64, cap=5.0, k_scale=3.0),
    "slopes": dict(lens=[100, 30], new=[60, 30], hk=2, group=2, d=64, slopes=True),
    "everything": dict(lens=[180, 70], new=[150, 70], hk=1, group=4, d=80, tpp=4, cap=20.0, slopes=True, window=50, prefix=[3, 9]),
    "many requests": dict(lens=[(i * 3) % 9 for i in range(140)], new=[(i * 3) % 9 for i in range(140)], hk=1, group=1, d=64),
    "few rows, long cache": dict(lens=[2500, 1300], new=[2, 5], hk=1, group=2, d=64, tpp=2),
}


def _offsets(new):
    return torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill(rt, name, dtype):
    spec = PREFILL[name]
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, name, spec, dtype, spec["new"])
    cache, kt, vt = c.to_gpu()
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets(spec["new"]), **dev)
    _check_attn(f"prefill {name} {dtype}", c, q, rows, ref, out, lse)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_masked_infinities_do_not_spread(rt, dtype):
    """Infinities and NaN in K and V reach the rows that see them and no other."""
    spec = dict(lens=[90, 150], new=[90, 70], hk=2, group=2, d=64, tpp=4, window=40)
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, "", spec, dtype, spec["new"])
    c.set_v(0, 50, float("inf"), head=1, dim=3)
    c.set_v(0, 60, float("-inf"), head=1, dim=3)  # rows that see both: NaN
    c.set_v(0, 89, float("nan"), head=0, dim=63)
    c.set_v(1, 149, float("inf"), head=0, dim=0)
    c.set_v(1, 20, float("nan"), head=1, dim=8)   # left behind by the window
    cache, kt, vt = c.to_gpu()
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets(spec["new"]), **dev)
    want, bound, _ = ku.attention(c, q, rows, **ref)
    assert torch.isinf(want).any() and torch.isnan(want).any()
    ku.check(out, want, bound, "prefill with infinities")
    # one token each: key 20 of request 1 and all of request 0 past its window unseen
    rows = [(0, 89), (1, 149)]
    last = torch.stack([q[89], q[159]])
    got = torch.empty(2, 4, 64, dtype=T[dtype], device="cuda")
    cache.decode(last.cuda(), got, kt, vt, seq, scale=ref["scale"], window=40)
    want, bound, _ = ku.attention(c, last, rows, **ref)
    ku.check(got, want, bound, "decode with infinities")


def test_minus_infinity_scores_and_nan_keys(rt):
    """Scores of minus infinity weigh nothing; a NaN key makes the rows that see it NaN."""
    c = ku.Cache(np.random.default_rng(6), [40, 40], dtype="f16", hk=1, d=64)
    for r, j, x in ((0, 39, float("-inf")), (1, 30, float("nan"))):
        c.k[r][j, 0, 0] = x
        c.pool[int(c.kt[r, j]), 0] = x
    q = _query(c, 1, 80, "f16").abs()
    rows = [(r, j) for r in range(2) for j in range(40)]
    cache, kt, vt = c.to_gpu()
    seq = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out = torch.empty(80, 1, 64, dtype=torch.float16, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets([40, 40]), scale=0.125)
    want, bound, _ = ku.attention(c, q, rows, scale=0.125)
    bound[torch.isnan(bound)] = 1.0
    assert int(torch.isnan(want[:, 0, 0]).sum()) == 10
    ku.check(out, want, bound, "prefill")
    got = torch.empty(2, 1, 64, dtype=torch.float16, device="cuda")
    cache.decode(q[[39, 79]].cuda(), got, kt, vt, seq, scale=0.125)
    ku.check(got, want[[39, 79]], bound[[39, 79]], "decode")


@pytest.mark.parametrize("group", [1, 4])
def test_bad_device_data(rt, group):
    """Page ids outside the pool read as NaN, lengths outside the table make NaN rows, rows of
    no request stay as they are; other requests are unharmed."""
    c = ku.Cache(np.random.default_rng(7), [40, 40, 40, 40, 40], dtype="bf16", hk=2, d=64, tpp=2)
    c.kt[1, 3], c.vt[2, 19] = -1, c.n_pages
    c.kt[1, 5] = 2147483647
    q = _query(c, 2 * group, 52, "bf16")
    cache, kt, vt = c.to_gpu()
    seq = torch.tensor([40, 40, 40, 43, -1], dtype=torch.int32, device="cuda")  # the table: 42 tokens
    assert c.max_blocks * 2 == 42
    out = torch.full((52, 2 * group, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets([10] * 5), scale=0.2)
    got = torch.full((5, 2 * group, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    last = q[[9, 19, 29, 39, 49]]
    cache.decode(last.cuda(), got, kt, vt, seq, scale=0.2)
    want, bound, _ = ku.attention(c, q[:10], [(0, 30 + i) for i in range(10)], scale=0.2)
    ku.check(out[:10], want, bound, "the request beside")
    ku.check(got[:1], want[9:], bound[9:], "the request beside, one token")
    assert torch.isnan(got[1:]).all() and torch.isnan(out[10:20]).all() and torch.isnan(out[30:50]).all()
    assert not torch.isnan(out[20:28]).any() and torch.isnan(out[28:30]).all()  # V page of positions 38, 39
    assert (out[50:] == 7).all()


def test_offsets_past_32_bits(rt):
    """Pages past 2^32 elements of the pool: written, then read back by both attentions."""
    hk, d, P = 8, 64, 8192
    n_pages = (1 << 32) // P + 4000
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * P:
        pytest.skip("not enough device memory")
    pool = torch.empty(n_pages * P, dtype=torch.bfloat16, device="cuda")
    cache = rt.KVCache(pool, n_pages, page_elems=P, dtype="bf16", n_kv_heads=hk, head_dim=d, tokens_per_page=16)
    n = 100
    g = torch.Generator().manual_seed(8)
    q, k, v = [torch.randn(n, hk, d, generator=g).bfloat16() for _ in range(3)]
    ids = torch.arange(n_pages - 14, n_pages, dtype=torch.int32, device="cuda")
    t = rt.KVTables(2, 1, 8, n)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.tables(t, ids, i32(0), i32(n))
    out = torch.empty(n, hk, d, dtype=torch.bfloat16, device="cuda")
    cache.write(q.cuda(), k.cuda(), v.cuda(), out, t.position, t.slots[0], t.slots[1])
    assert torch.equal(out.cpu(), q)
    c = ku.Cache(np.random.default_rng(0), [0], dtype="bf16", hk=hk, d=d)
    c.lens, c.k, c.v = [n], [k], [v]
    cache.prefill(out, out, t.table[0], t.table[1], t.seq_len, t.q_offsets, scale=0.125)
    want, bound, _ = ku.attention(c, q, [(0, i) for i in range(n)], scale=0.125)
    ku.check(out, want, bound, "prefill")
    got = torch.empty(1, hk, d, dtype=torch.bfloat16, device="cuda")
    cache.decode(q[-1:].cuda(), got, t.table[0], t.table[1], t.seq_len, scale=0.125)
    ku.check(got, want[-1:], bound[-1:], "decode")


def test_other_stream_and_graph(rt):
    """A decode step (tables, write, attention) on a side stream, and captured: replays with
    other lengths and inputs equal the eager calls bit for bit."""
    hk, group, d, tpp, R, width = 2, 2, 64, 2, 3, 40
    hq, planes = hk * group, 2
    n_pages = 2 * R * width
    g = torch.Generator().manual_seed(9)
    pool0 = torch.randn(n_pages * tpp * hk * d, generator=g).half().cuda()
    ids = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    rope = rt.Rope(d)
    dev = "cuda"
    past, new = torch.zeros(R, dtype=torch.int32, device=dev), torch.zeros(R, dtype=torch.int32, device=dev)
    q, k, v = (torch.empty(R, h, d, dtype=torch.float16, device=dev) for h in (hq, hk, hk))
    x, y, z = (torch.empty(R, hq, d, dtype=torch.float16, device=dev) for _ in range(3))
    pool = pool0.clone()
    cache = rt.KVCache(pool, n_pages, page_elems=tpp * hk * d, dtype="f16", n_kv_heads=hk, head_dim=d, tokens_per_page=tpp)
    t = rt.KVTables(planes, R, width, R)
    side = torch.cuda.Stream()

    def bind(stream):
        args = (t.table[0], t.table[1], t.seq_len)
        return [cache.bind_tables(t, ids, past, new, stream=stream),
                cache.bind_write(q, k, v, x, t.position, t.slots[0], t.slots[1], rope=rope, norm=True, stream=stream),
                cache.bind_decode(x, y, *args, stream=stream),
                cache.bind_prefill(x, z, *args, t.q_offsets, stream=stream)]

    def fill(seed):
        h = torch.Generator().manual_seed(seed)
        lens = torch.randint(0, width * tpp - 1, (R,), generator=h, dtype=torch.int32)
        past.copy_(lens)
        new.fill_(1)
        for a in (q, k, v):
            a.copy_(torch.randn(a.shape, generator=h))
        pool.copy_(pool0)

    eager = bind(None)
    fill(0)
    for call in eager:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in bind(None):
            call()
    for seed in range(1, 5):
        fill(seed)
        for call in eager:
            call()
        want = [a.clone() for a in (pool, y, z, t.table, t.slots)]
        for a in (y, z):
            a.zero_()
        fill(seed)
        graph.replay()
        for a, b in zip((pool, y, z, t.table, t.slots), want):
            assert torch.equal(a, b)
        fill(seed)
        for a in (y, z):
            a.zero_()
        side.wait_stream(torch.cuda.current_stream())
        for call in bind(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((pool, y, z, t.table, t.slots), want):
            assert torch.equal(a, b)
    assert torch.allclose(y.float(), z.float(), rtol=2e-2, atol=2e-2)


def test_timing_records_each_operator(rt):
    from heterogeneous_lora_amd import _lib
    c = ku.Cache(np.random.default_rng(1), [5], hk=1, d=64)
    cache, kt, vt = c.to_gpu()
    q = _query(c, 1, 1, "f16").cuda()
    seq = torch.tensor([5], dtype=torch.int32, device="cuda")
    _lib.timing_read_all()
    _lib.timing_enable(True)
    cache.decode(q, q.clone(), kt, vt, seq)
    cache.prefill(q, q.clone(), kt, vt, seq, _offsets([1]))
    _lib.timing_enable(False)
    names, ms = _lib.timing_read_all()
    assert names == ["attn_decode", "attn_prefill"] and (ms > 0).all()
