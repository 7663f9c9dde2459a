"""The cache in 4 bits where it can go wrong: groups at the edges of the format, slots and pages
outside the pool, values that are no numbers, lengths out of range, workspaces with other contents,
graphs and streams, large pools."""

import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util
from heterogeneous_lora_amd import _lib, runtime
from test_gpu_kv4 import check_bytes, long_table, written

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- write and read

def edges(q, k, v):
    """Every kind of group, in K and V alike (the same for host and device tensors)."""
    n, h, d = k.shape
    x = torch.zeros(n, h, d)
    j = torch.arange(d)
    x[0] = (j % 16 - 8) / 4                              # quarters: ties between levels of step 1/3
    x[1] = torch.where(j % 32 == 0, 6.0, (j % 16 - 8) / 4.0)   # step 1: ties between levels
    x[2] = 60000.0                                       # near the largest of f16
    x[3] = 0.0
    x[4] = -0.0
    x[5] = 2.0 ** -24 * (j % 5)                          # f16's smallest
    x[6] = torch.where(j == 3, math.inf, 1.0)
    x[7] = torch.where(j == 7, math.nan, 1.0)
    x[8] = torch.where(j % 32 == 31, -math.inf, 2.0)
    x[9] = 6 * (1 + (2 * (j % 8) + 1) / 16.0)            # each group's largest ties between two steps
    x[10] = 6 * (1 + (2 * h + 1) / 16.0) * (1 + torch.where(j % 32 == 0, 2.0 ** -8, -2.0 ** -8))
    x[11] = 2.0 ** -17 * (j % 7)                         # around the smallest steps
    x[12] = 3 * 2.0 ** -17 * (1 + j % 2)                 # half the smallest step times 6, and that times 6
    for t in (k, v):
        t[:13] = x[:13].to(t.dtype).to(t.device)
    if k.dtype == torch.bfloat16:
        for t in (k, v):
            t[13] = 3e38 * (1 - 2 * (j % 2)).to(t.device)
            t[14] = (1e-40 * j).to(t.device)
            t[15] = (61440.0 * (1 + (j % 3) / 16.0)).to(t.device)  # around what steps end at


@pytest.mark.parametrize("dtype,hk,d,tpp", [("f16", 2, 128, 3), ("bf16", 3, 96, 1), ("f16", 1, 40, 2), ("bf16", 2, 256, 5)])
def test_groups_at_the_edges(dtype, hk, d, tpp):
    cache, pool, slots, dev_slots, _, _, want, lay = written(dtype, hk, hk, d, tpp, 24, rotary=0, seed=3, bend=edges)
    check_bytes(cache, pool, slots, want, lay, tpp)
    k, v = (torch.empty(24, hk, d, dtype=util.TORCH[dtype], device="cuda") for _ in range(2))
    cache.read(k, v, *dev_slots)
    for got, x in ((k, want[0]), (v, want[1])):
        ref = four.values(*four.held(x), d)
        got = got.cpu().double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and int(torch.isnan(ref).sum()) > 0
        assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(ref, nan=0.0))


@pytest.mark.parametrize("interleaved", [False, True])
def test_many_keys_decide_as_64_bits(interleaved):
    """Some millions of rotated and normalised values: each on its own side of the borders."""
    cache, pool, slots, _, _, _, want, lay = written("bf16", 8, 8, 128, 15, 3000, rotary=128, interleaved=interleaved,
                                                     norm=True, seed=12)
    check_bytes(cache, pool, slots, want, lay, 15)


def test_rows_without_a_place_change_nothing():
    hk, d, tpp, n = 2, 64, 3, 8
    size = four.layout(hk, d)[2]
    P = tpp * size // 2
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, h, d, generator=g).half().cuda() for h in (4, hk, hk))
    pool = torch.randint(0, 256, (5, 2 * P), generator=g, dtype=torch.uint8).cuda()
    before = pool.clone()
    cache = runtime.KVCache(pool, 5, page_elems=P, dtype="f16", n_kv_heads=hk, head_dim=d, tokens_per_page=tpp, bits=4)
    out = torch.full((n, 4, d), 7.0, dtype=torch.float16, device="cuda")
    bad = torch.tensor([-1, 15, 1 << 31, 1 << 40, -(1 << 60), (1 << 63) - 1, 16, -2], device="cuda")
    cache.write(q, k, v, out, i32([0, -1, 2, 3, 4, -5, 6, 7]), bad, bad)
    assert torch.equal(pool, before)
    skipped = torch.tensor([0, 1, 0, 0, 0, 1, 0, 0], dtype=torch.bool, device="cuda")
    assert bool((out[skipped] == 7.0).all()) and torch.equal(out[~skipped], q[~skipped])
    # negative positions with good slots store nothing either; k alone may have a place
    at = torch.arange(n, device="cuda")
    cache.write(q, k, v, out, i32([-1] * n), at, at)
    assert torch.equal(pool, before)
    cache.write(q, k, v, out, i32([0] * n), at, bad)
    cache.write(q, k, v, out, i32([0] * n), bad, at + 7)
    want = four.values(*four.held(torch.cat([k[:7], v]).cpu().double()), d)
    got = torch.full((15, hk, d + 8), 9.0, dtype=torch.float16, device="cuda")
    cache.read(got[..., :d], None, torch.arange(15, device="cuda"), None)
    assert torch.equal(got[..., :d].cpu().double(), want) and bool((got[..., d:] == 9.0).all())
    # reads of no place leave their rows
    rows = torch.full((n, hk, d), 7.0, dtype=torch.float16, device="cuda")
    both = bad.clone()
    both[4] = 2
    cache.read(None, rows, None, both)
    assert torch.equal(rows[4].cpu().double(), want[2])
    rows[4] = 7.0
    assert bool((rows == 7.0).all())


def test_strided_rows():
    """q, k, v as parts of one projection, outputs with gaps, the same token twice."""
    hk, d, n = 2, 96, 9
    size = four.layout(hk, d)[2]
    pool = torch.zeros(n, size, dtype=torch.uint8, device="cuda")
    cache = runtime.KVCache(pool, n, page_elems=size // 2, dtype="bf16", n_kv_heads=hk, head_dim=d, bits=4)
    g = torch.Generator().manual_seed(2)
    packed = torch.randn(n, 3 * hk, d, generator=g).bfloat16().cuda()
    q, k, v = packed.split(hk, 1)
    q, k, v = q.transpose(0, 1).contiguous().transpose(0, 1), k, v
    out = torch.zeros(n, 2 * hk, d + 8, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(n, device="cuda")
    cache.write(q, k, v, out[:, ::2, :d], i32([0] * n), at, torch.full_like(at, -1))
    assert torch.equal(out[:, ::2, :d], q) and bool((out[:, 1::2] == 0).all()) and bool((out[..., d:] == 0).all())
    to = torch.zeros(2 * n, 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    cache.read(to[::2, hk:], None, at.flip(0).contiguous(), None)
    cache.read(to[1::2, :hk], None, torch.full_like(at, 4), None)
    want = four.values(*four.held(k.cpu().double()), d)
    assert torch.equal(to[::2, hk:].cpu().double(), want.flip(0)) and bool((to[::2, :hk] == 0).all())
    assert torch.equal(to[1::2, :hk].cpu().double(), want[4].expand(n, hk, d)) and bool((to[1::2, hk:] == 0).all())


# ---------------------------------------------------------------- attention

def call(c, op, q, lens, *, new=None, ws=None, lse=None, **kw):
    cache, kt, vt = c.to_gpu()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    if op == "decode":
        cache.decode(q.cuda(), out, kt, vt, i32(lens), ws=ws, lse=lse, **kw)
    else:
        offsets = i32([0] + list(np.cumsum(new)))
        cache.prefill(q.cuda(), out, kt, vt, i32(lens), offsets, ws=ws, lse=lse, **kw)
    return out


def close(got, ref, bound, what):
    """Within the bound where the reference is a number, no number where it is none."""
    got = got.cpu().double()
    none = ~torch.isfinite(ref.out)
    assert torch.equal(~torch.isfinite(got), none), f"{what}: {int((~torch.isfinite(got) != none).sum())} places"
    util.check(got[~none], ref.out[~none], bound[~none], what)


WAYS = ["few", "many", "straight", "back"]  # decode of few keys, of many; prefill from the codes, read back


def make(way, rng, lens, dtype, d=64, hk=2, tpp=3, hq=4):
    """Cache, q, rows and the call's kind for one of WAYS."""
    if way in ("few", "many"):
        c = four.Cache(rng, lens, dtype=dtype, hk=hk, d=d, tpp=tpp, blocks_more=long_table(hk, len(lens), tpp) if way == "many" else 1)
        return c, hq, [1] * len(lens), "decode"
    c = four.Cache(rng, lens, dtype=dtype, hk=hk, d=d, tpp=tpp)
    new = [min(n, 70 if way == "back" else 40) for n in lens]
    if way == "back":  # (4096 rows a request and KV head)
        hq = hk * (64 if sum(new) * 64 >= 4096 * len(lens) else 128)
        assert sum(new) * hq // hk >= 4096 * len(lens)
    return c, hq, new, "prefill"


def rows_of(lens, new):
    return [(r, n - m + i) for r, (n, m) in enumerate(zip(lens, new)) for i in range(m)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("way,window", [(w, n) for w in WAYS for n in (0, 40) if (w, n) != ("many", 40)])  # (a window: few)
def test_no_numbers_reach_the_rows_that_see_them(way, dtype, window):
    rng = np.random.default_rng(31)
    lens = [150, 75, 90]
    c, hq, new, op = make(way, rng, lens, dtype)

    def spoil(r, token, which, head, dim, value):
        x = (c.k, c.v)[which][r][token].double()[None].clone()
        x[0, head, dim] = value
        c.put(r, slice(token, token + 1), which, x)
    spoil(0, 147, 1, 0, 40, math.nan)    # seen by the last rows of request 0, V, dims 32 .. 63 of head 0
    spoil(0, 2, 1, 1, 5, math.inf)       # outside a window
    spoil(1, 74, 0, 1, 3, -math.inf)     # K: all of head 1's row
    spoil(2, 3, 0, 0, 3, math.nan)       # outside a window
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64))).to(util.TORCH[dtype])
    got = call(c, op, q, lens, new=new, window=window)
    ref = four.attention(c, q, rows_of(lens, new), scale=0.125, window=window)
    assert bool(torch.isnan(ref.out).any()) and bool(torch.isfinite(ref.out).any())
    close(got, ref, four.bound(ref, dtype, op == "decode", back=way == "back"), way)


@pytest.mark.parametrize("way", WAYS)
def test_nothing_of_other_tokens_is_read(way):
    """Pages' other places, pages of no request and the tables' rest hold steps that are no numbers
    (four.Cache); here the workspace too."""
    rng = np.random.default_rng(32)
    lens = [1, 129, 0, 64, 65]
    c, hq, new, op = make(way, rng, lens, "f16", tpp=7)
    c.kt[:, -1] = 1 << 30
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64))).half()
    cache, kt, vt = c.to_gpu()
    a = _lib.Attn(n_q_heads=hq)
    size = cache.workspace_size(cache._kv(len(lens), c.max_blocks), a, 0 if op == "decode" else sum(new))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    ws[:10240] = 0
    before = ws[:10240].clone()
    got = call(c, op, q, lens, new=new, ws=ws)
    rows = [(r, n - 1) for r, n in enumerate(lens)] if op == "decode" else rows_of(lens, new)
    ref = four.attention(c, q, rows, scale=0.125)
    util.check(got, ref.out, four.bound(ref, "f16", op == "decode", back=way == "back"), way)
    assert torch.equal(ws[:10240], before)


@pytest.mark.parametrize("way", WAYS)
def test_pages_and_lengths_out_of_range(way):
    rng = np.random.default_rng(33)
    lens = [100, 90, 80, 70]
    c, hq, new, op = make(way, rng, lens, "bf16", hk=1, tpp=4)
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64))).bfloat16()
    c.vt[1, 22] = c.n_pages       # the last rows of request 1 see keys 88, 89 there
    c.kt[2, 19] = -1 << 31        # request 2: keys 76 .. 79
    for r, first, which in ((1, 88, 1), (2, 76, 0)):
        (c.k, c.v)[which][r][first:] = math.nan
    got = call(c, op, q, lens, new=new)
    ref = four.attention(c, q, rows_of(lens, new), scale=0.125)
    assert bool(torch.isnan(ref.out).any()) and bool(torch.isfinite(ref.out).any())
    bound = four.bound(ref, "bf16", op == "decode", back=way == "back")
    close(got, ref, bound, way)
    # lengths outside the table: that request's rows alone
    for bad in (-1, c.max_blocks * 4 + 1, 2 ** 31 - 1, -2 ** 31):
        lse = torch.zeros(sum(new), hq, device="cuda")
        seq = lens[:3] + [bad]
        again = call(c, op, q, seq, new=new, lse=lse)
        m = sum(new[:3])
        close(again[:m], SimpleNamespace(out=ref.out[:m]), bound[:m], way)
        assert bool(torch.isnan(again[m:]).all()) and bool(torch.isnan(lse[m:]).all())


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("size", [2.0 ** 90, 2.0 ** -100, "mixed"])
def test_bf16_queries_of_any_size(way, size):
    """Rows are brought into f16's range by powers of two of their own; scale takes them back."""
    rng = np.random.default_rng(34)
    lens = [60, 131]
    c, hq, new, op = make(way, rng, lens, "bf16")
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64)))
    scale = 0.125
    if size == "mixed":  # the last rows and heads larger than the others, some small dimensions, a row of zeros
        q[:, 1] *= 8
        q[..., 5] *= 2.0 ** -12
        q[0, 0] = 0
    else:
        q, scale = q * size, 0.125 / size
    q = q.bfloat16()
    got = call(c, op, q, lens, new=new, scale=scale)
    ref = four.attention(c, q, rows_of(lens, new), scale=scale)
    util.check(got, ref.out, four.bound(ref, "bf16", op == "decode", back=way == "back"), way)


@pytest.mark.parametrize("way", WAYS)
def test_strides_and_unaligned_rows(way):
    rng = np.random.default_rng(35)
    lens = [40, 100]
    c, hq, new, op = make(way, rng, lens, "f16", d=72, tpp=2)
    n = sum(new)
    q = torch.from_numpy(rng.standard_normal((n, hq, 72))).half()
    wide = torch.full((hq, n, 88), 7.0, dtype=torch.float16, device="cuda")
    out = wide.transpose(0, 1)[..., 8:80]
    store = torch.zeros(n, hq, 96, dtype=torch.float16, device="cuda")
    qd = store[..., 16:88]
    qd.copy_(q)
    cache, kt, vt = c.to_gpu()
    if op == "decode":
        cache.decode(qd, out, kt, vt, i32(lens))
    else:
        cache.prefill(qd, out, kt, vt, i32(lens), i32([0] + list(np.cumsum(new))))
    ref = four.attention(c, q, rows_of(lens, new), scale=72 ** -0.5)
    util.check(out, ref.out, four.bound(ref, "f16", op == "decode", back=way == "back"), way)
    assert bool((wide[..., :8] == 7.0).all()) and bool((wide[..., 80:] == 7.0).all())


@pytest.mark.parametrize("way", ["straight", "back"])
def test_offsets_outside_the_rows(way):
    """q_offsets that are negative, fall or pass the last row: rows of no request stay as they were."""
    rng = np.random.default_rng(36)
    lens = [90, 80, 70]
    c, hq, new, _ = make(way, rng, lens, "f16")
    n = sum(new)
    q = torch.from_numpy(rng.standard_normal((n, hq, 64))).half()
    cache, kt, vt = c.to_gpu()
    for offsets in ([-5, new[0], new[0], new[0] + 20], [0, new[0], 10, 10 ** 9]):
        out = torch.full((n, hq, 64), 7.0, dtype=torch.float16, device="cuda")
        cache.prefill(q.cuda(), out, kt, vt, i32(lens), i32(offsets))
        if offsets[0] < 0:
            rows = rows_of([lens[0], lens[2]], [new[0], 20])
            rows = [((0, 2)[r], p) for r, p in rows]
            ref = four.attention(c, q[:len(rows)], rows, scale=0.125)
            util.check(out[:len(rows)], ref.out, four.bound(ref, "f16", False), way)
            assert bool((out[len(rows):] == 7.0).all())
        else:
            ref = four.attention(c, q[:10], [(0, lens[0] - new[0] + i) for i in range(10)], scale=0.125)
            util.check(out[:10], ref.out, four.bound(ref, "f16", False), way)
            assert bool(torch.isfinite(out).all())


# ---------------------------------------------------------------- graphs, streams, sizes

def test_replays_with_one_workspace():
    """Calls of every way, and of a cache in 16 bits, in one captured graph and one workspace, replayed
    with other lengths and with eager calls in that workspace between."""
    import attn_exact as ax
    rng = np.random.default_rng(40)
    full = [900, 2000, 640]
    few = four.Cache(rng, full, dtype="bf16", hk=2, d=128, tpp=4)
    many = four.Cache(rng, full, dtype="bf16", hk=2, d=128, tpp=4, blocks_more=long_table(2, 3, 4))
    plain = ax.dense_cache(full, dtype="bf16", hk=2, d=128, tpp=4, seed=41)
    g = torch.Generator().manual_seed(42)
    q4 = torch.randn(9, 4, 128, generator=g).bfloat16().cuda()
    wide = torch.randn(200, 128, 128, generator=g).bfloat16().cuda()
    seq, offsets, woff = i32(full), i32([0, 1, 4, 9]), i32([0, 70, 130, 200])
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    caches = [x.to_gpu() for x in (few, many)] + [ax.to_gpu(plain)]
    outs = lambda: [torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in caches] + \
        [torch.empty_like(q4) for _ in range(2)] + [torch.empty_like(wide)]

    def bind(o):
        calls = [cache.bind_decode(q4[:3], o[i], kt, vt, seq, ws=ws) for i, (cache, kt, vt) in enumerate(caches)]
        for i, at in ((3, 0), (4, 2)):
            cache, kt, vt = caches[at]
            calls.append(cache.bind_prefill(q4, o[i], kt, vt, seq, offsets, ws=ws))
        cache, kt, vt = caches[0]
        calls.append(cache.bind_prefill(wide, o[5], kt, vt, seq, woff, ws=ws))
        return calls
    x, y = outs(), outs()
    eager = bind(x)
    for run in eager:
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for run in bind(y):
            run()
    for turn, lens in enumerate([full, [10, 1999, 300], [0, 70, 640], [77, 1, 2], full]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        q4.copy_(torch.randn(9, 4, 128, generator=g))
        wide.copy_(torch.randn(200, 128, 128, generator=g))
        for t in y:
            t.fill_(7.0)
        for i, run in enumerate(eager):
            run()
        graph.replay()
        for run in eager[::-1]:
            run()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(x, y)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), (turn, lens, i)
    assert int(ws[:10240].view(torch.int32).abs().max()) == 0


def test_captured_write_and_read():
    cache, pool, slots, dev_slots, out, (q, position, kw), want, lay = written("f16", 2, 4, 64, 3, 20, rotary=64, seed=5)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(20, 2, 64, generator=g).half().cuda() for _ in range(2))
    back = [torch.empty_like(k) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    write = lambda: cache.write(q, k, v, out, position, *dev_slots, **kw)
    write()
    cache.read(*back, *dev_slots)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        write()
        cache.read(*back, *dev_slots)
    for _ in range(4):
        k.copy_(torch.randn(20, 2, 64, generator=g))
        v.copy_(torch.randn(20, 2, 64, generator=g))
        cache.pool.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        y, _ = util.written(k.cpu(), position.cpu(), kw["rope"].turns_host, interleaved=False, cos_sin_scale=1.25,
                            norm=False, eps=0.0, weight=None)
        assert torch.equal(back[0].cpu().double(), four.values(*four.held(y), 64))
        assert torch.equal(back[1].cpu().double(), four.values(*four.held(v.cpu()), 64))


@pytest.mark.parametrize("way", WAYS)
def test_on_another_stream(way):
    """Work of a stream of its own: its workspace is made and zeroed in that stream's order."""
    rng = np.random.default_rng(45)
    lens = [700, 90]
    c, hq, new, op = make(way, rng, lens, "f16")
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64))).half()
    want = call(c, op, q, lens, new=new)
    torch.cuda.synchronize()
    cache, kt, vt = c.to_gpu()
    side, dq, seq, offsets = torch.cuda.Stream(), q.cuda(), i32(lens), i32([0] + list(np.cumsum(new)))
    for _ in range(3):
        got = torch.full_like(want, 7.0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.full((64 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
        x = torch.randn(2048, 2048, device="cuda")
        for _ in range(20):
            x = x @ x / 64
        if op == "decode":
            cache.decode(dq, got, kt, vt, seq, stream=side)
        else:
            cache.prefill(dq, got, kt, vt, seq, offsets, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """The same cache read by two calls at once, each with its workspace."""
    rng = np.random.default_rng(46)
    lens = [3000, 2000]
    c, hq, new, _ = make("many", rng, lens, "bf16")
    q = [torch.from_numpy(rng.standard_normal((2, hq, 64))).bfloat16() for _ in range(2)]
    want = [call(c, "decode", x, lens) for x in q]
    cache, kt, vt = c.to_gpu()
    streams, dq, seq = [torch.cuda.Stream() for _ in range(2)], [x.cuda() for x in q], i32(lens)
    got = [torch.full_like(w, 7.0) for w in want]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    runs = [cache.bind_decode(x, o, kt, vt, seq, stream=s) for x, o, s in zip(dq, got, streams)]
    for _ in range(20):
        for run in runs:
            run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("way", WAYS)
def test_pages_past_4_gib(way):
    """Offsets of pages, of slots and of queries' rows above 32 bits."""
    rng = np.random.default_rng(47)
    lens = [90, 140]
    c, hq, new, op = make(way, rng, lens, "f16", tpp=2)
    far = 5 * (1 << 30) // (2 * c.P)  # pages
    pool = torch.empty(far + c.n_pages, 2 * c.P, dtype=torch.uint8, device="cuda")
    pool[far:] = c.pool.cuda()
    cache = runtime.KVCache(pool, far + c.n_pages, page_elems=c.P, dtype="f16", n_kv_heads=2, head_dim=64, tokens_per_page=2,
                            bits=4)
    move = lambda t: torch.from_numpy(np.where(t >= 0, t + far, t).astype(np.int32)).cuda()
    kt, vt = move(c.kt), move(c.vt)
    q = torch.from_numpy(rng.standard_normal((sum(new), hq, 64))).half()
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    if op == "decode":
        cache.decode(q.cuda(), out, kt, vt, i32(lens))
    else:
        cache.prefill(q.cuda(), out, kt, vt, i32(lens), i32([0] + list(np.cumsum(new))))
    ref = four.attention(c, q, rows_of(lens, new), scale=0.125)
    util.check(out, ref.out, four.bound(ref, "f16", op == "decode", back=way == "back"), way)
    if way == "few":  # write and read there too
        x = torch.from_numpy(rng.standard_normal((4, 2, 64))).half().cuda()
        at = (torch.arange(4, device="cuda") + 2 * far)
        cache.write(x, x, x, torch.empty_like(x), i32([0] * 4), at, at + 4)
        got = [torch.empty_like(x) for _ in range(2)]
        cache.read(*got, at, at + 4)
        want = four.values(*four.held(x.cpu()), 64)
        assert all(torch.equal(y.cpu().double(), want) for y in got)


@pytest.mark.parametrize("longest", [100, 700])
def test_decode_of_16384_requests(longest):
    """The most requests: with a short table few keys, with a longer one spans over all of them."""
    lens = [i % 5 for i in range(16384)]
    lens[77], lens[16383] = longest, longest - 30
    rng = np.random.default_rng(48)
    some = [0, 1, 4, 76, 77, 78, 511, 8191, 16383]
    c = four.Cache(rng, [lens[r] for r in some], dtype="f16", hk=1, d=8, tpp=4)
    kt, vt = (np.full((16384, c.max_blocks), -1, np.int32) for _ in range(2))
    kt[:, 0], vt[:, 0] = c.kt[4, 0], c.vt[4, 0]  # (the others see that request's first tokens)
    kt[some], vt[some] = c.kt, c.vt
    cache, _, _ = c.to_gpu()
    q = torch.randn(16384, 2, 8, generator=torch.Generator().manual_seed(4)).half()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    cache.decode(q.cuda(), out, torch.from_numpy(kt).cuda(), torch.from_numpy(vt).cuda(), i32(lens), scale=0.3)
    ref = four.attention(c, q[some], [(i, n - 1) for i, n in enumerate(c.lens)], scale=0.3)
    util.check(out[some], ref.out, four.bound(ref, "f16", True), "decode")
    empty = torch.tensor(lens) == 0
    assert bool((out.cpu()[empty] == 0).all())
    assert bool((out != 7.0).any(-1).any(-1).all())


@pytest.mark.parametrize("op", ["decode", "prefill"])
@pytest.mark.parametrize("window,prefix", [(1000, 0), (700, 300)])
def test_2_to_the_30_tokens(op, window, prefix):
    """A request as long as a table allows, its blocks on two pages: the first, and all others."""
    d, tpp, blocks = 8, 1 << 18, 1 << 12
    n = (1 << 30) - 5
    rng = np.random.default_rng(49)
    c = four.Cache(rng, [tpp, tpp], dtype="f16", hk=1, d=d, tpp=tpp, extra=0)
    table = lambda t: i32([[int(t[0, 0])] + [int(t[1, 0])] * (blocks - 1)])
    cache, _, _ = c.to_gpu()
    rows = 1 if op == "decode" else 3
    q = torch.randn(rows, 2, d, generator=torch.Generator().manual_seed(5)).half()
    out = torch.empty(rows, 2, d, dtype=torch.float16, device="cuda")
    opts = dict(scale=0.3, window=window, prefix_len=i32([prefix]) if prefix else None)
    if op == "decode":
        cache.decode(q.cuda(), out, table(c.kt), table(c.vt), i32([n]), **opts)
    else:
        cache.prefill(q.cuda(), out, table(c.kt), table(c.vt), i32([n]), i32([0, rows]), **opts)
    for i in range(rows):
        p = n - rows + i
        j = np.arange(p - window + 1, p + 1) % tpp
        k, v = (torch.cat([x[0][:prefix], x[1][j]]) for x in (c.k, c.v))
        one = SimpleNamespace(hk=1, lens=[len(k)], k=[k], v=[v])
        ref = four.attention(one, q[i:i + 1], [(0, len(k) - 1)], scale=0.3)
        util.check(out[i:i + 1], ref.out, four.bound(ref, "f16", op == "decode"), f"{op} row {i}")


@pytest.mark.parametrize("way", ["few", "many", "straight"])
@pytest.mark.parametrize("hk,group,d", [(1024, 1, 8), (1024, 16, 8), (521, 3, 40), (1, 4096, 64), (63, 5, 136), (17, 17, 256)])
def test_many_heads(way, hk, group, d):
    """As many heads as there may be, odd numbers of them, steps that begin anywhere in 16 bytes."""
    rng = np.random.default_rng(hk + group)
    lens = [70, 3]
    c = four.Cache(rng, lens, dtype="bf16", hk=hk, d=d, tpp=1, blocks_more=long_table(hk, 2, 1) if way == "many" else 1)
    op = "prefill" if way == "straight" else "decode"
    new = [2, 1] if op == "prefill" else [1, 1]
    q = torch.from_numpy(rng.standard_normal((sum(new), hk * group, d))).bfloat16()
    got = call(c, op, q, lens, new=new)
    ref = four.attention(c, q, rows_of(lens, new), scale=d ** -0.5)
    back = op == "prefill" and 3 * group >= 2 * 4096
    util.check(got, ref.out, four.bound(ref, "bf16", op == "decode", back=back), way)


@pytest.mark.parametrize("hk,hq,d", [(1024, 2048, 8), (521, 1, 40), (1, 300, 256)])
def test_write_of_many_heads(hk, hq, d):
    cache, pool, slots, dev_slots, _, _, want, lay = written("f16", hk, hq, d, 1, 5, rotary=8, norm=True, seed=8)
    check_bytes(cache, pool, slots, want, lay, 1)
    k, v = (torch.empty(5, hk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    cache.read(k, v, *dev_slots)
    for got, x in ((k, want[0]), (v, want[1])):
        assert torch.equal(got.cpu().double(), four.values(*four.held(x), d))
