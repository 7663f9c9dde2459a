"""The cache in 4 bits on the GPU against 64-bit references: bytes stored, values read, attention."""

import math

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util
from heterogeneous_lora_amd import runtime

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- write and read

def written(dtype, hk, hq, d, tpp, n, *, rotary, interleaved=False, norm=False, weights=True, seed=0, pad=0, bend=None):
    """One write of n tokens: the pool before and after, slots, q out, and what K and V should be."""
    rng = np.random.default_rng(seed)
    g, sb, size = four.layout(hk, d)
    P = -(-tpp * size // 16) * 8 + 8
    n_pages = 2 * (-(-n // tpp) + 1)
    gen = torch.Generator().manual_seed(seed)
    kind = util.TORCH[dtype]
    packed = (torch.randn(n, (hq + 2 * hk) * (d + pad), generator=gen)).to(kind)
    q, k, v = (x.unflatten(1, (-1, d + pad))[..., :d] for x in packed.split([m * (d + pad) for m in (hq, hk, hk)], 1))
    if bend:
        bend(q, k, v)
    order = rng.permutation(n_pages)
    slots = [np.concatenate([order[i::2]])[np.arange(n) // tpp].astype(np.int64) * tpp + np.arange(n) % tpp
             for i in range(2)]
    position = rng.integers(0, 1 << 20, n).astype(np.int32)
    qw, kw = ((1 + 0.2 * torch.randn(d, generator=gen)).to(kind) if norm and weights else None for _ in range(2))
    pool = torch.from_numpy(rng.integers(0, 256, (n_pages, 2 * P), dtype=np.uint8))
    rope = runtime.Rope(rotary, interleaved=interleaved, cos_sin_scale=1.25) if rotary else None
    cache = runtime.KVCache(pool.cuda(), n_pages, page_elems=P, dtype=dtype, n_kv_heads=hk, head_dim=d,
                            tokens_per_page=tpp, bits=4)
    dev = packed.cuda()
    qd, kd, vd = (x.unflatten(1, (-1, d + pad))[..., :d] for x in dev.split([m * (d + pad) for m in (hq, hk, hk)], 1))
    if bend:
        bend(qd, kd, vd)
    out = torch.zeros(n, hq, d, dtype=kind, device="cuda")
    kw_args = dict(rope=rope, norm=norm, q_weight=None if qw is None else qw.cuda(),
                   k_weight=None if kw is None else kw.cuda(), eps=2.0 ** -20)
    ks, vs = (torch.from_numpy(x).cuda() for x in slots)
    cache.write(qd, kd, vd, out, torch.from_numpy(position).cuda(), ks, vs, **kw_args)
    turns = [] if rope is None else rope.turns_host
    want, _ = util.written(k, torch.from_numpy(position), turns, interleaved=interleaved, cos_sin_scale=1.25,
                           norm=norm, eps=2.0 ** -20, weight=kw)
    return cache, pool, slots, (ks, vs), out, (qd, torch.from_numpy(position).cuda(), kw_args), (want, v.double()), (g, sb, size)


def check_bytes(cache, pool, slots, want, lay, tpp):
    after = cache.pool.cpu().to(torch.int64)
    expect = pool.to(torch.int64).clone()
    g, sb, size = lay
    for at, x in zip(slots, want):
        raw = four.token_bytes(*four.held(x), sb)
        cols = torch.from_numpy((at % tpp)[:, None] * size + np.arange(size))
        page = torch.from_numpy(at // tpp)[:, None]
        expect[page, cols] = torch.where(raw < 0, after[page, cols], raw)
    assert torch.equal(after, expect), f"{int((after != expect).sum())} bytes differ"


SHAPES = [("f16", 4, 4, 64, 1), ("bf16", 8, 32, 128, 15), ("f16", 1, 8, 80, 7), ("bf16", 2, 2, 96, 2),
          ("f16", 3, 3, 256, 1), ("bf16", 5, 10, 40, 3), ("f16", 2, 4, 8, 5), ("bf16", 1, 1, 160, 4),
          ("f16", 2, 2, 72, 1), ("bf16", 4, 4, 32, 9), ("f16", 1, 1, 224, 2), ("f16", 2, 6, 192, 1)]


@pytest.mark.parametrize("dtype,hk,hq,d,tpp", SHAPES)
@pytest.mark.parametrize("rotary,interleaved,norm", [(0, False, False), (1, False, True), (1, True, False), (2, False, False), (2, True, True)])
def test_write_and_read(dtype, hk, hq, d, tpp, rotary, interleaved, norm):
    rotary = {0: 0, 1: d, 2: max(d // 16 * 8, 8)}[rotary]
    n = 37
    cache, pool, slots, dev_slots, out, rest, want, lay = written(dtype, hk, hq, d, tpp, n, rotary=rotary,
                                                                  interleaved=interleaved, norm=norm, seed=d + n, pad=8)
    check_bytes(cache, pool, slots, want, lay, tpp)
    k, v = (torch.full((n, hk, d), 9.0, dtype=util.TORCH[dtype], device="cuda") for _ in range(2))
    cache.read(k, v, *dev_slots)
    for got, x in ((k, want[0]), (v, want[1])):
        code, step = four.held(x)
        assert torch.equal(got.cpu().double(), four.values(code, step, d))
    # q as the write of 16 bits makes it
    qd, position, kw = rest
    plain = runtime.KVCache(torch.zeros(1, hk * d * tpp, dtype=torch.int16, device="cuda"), 1, page_elems=hk * d * tpp,
                            dtype=dtype, n_kv_heads=hk, head_dim=d, tokens_per_page=tpp)
    same = torch.zeros_like(out)
    plain.write(qd, None, None, same, position, None, None, **kw)
    ref, size = util.written(qd.cpu(), position.cpu(), [] if kw["rope"] is None else kw["rope"].turns_host,
                             interleaved=interleaved, cos_sin_scale=1.25, norm=norm, eps=2.0 ** -20,
                             weight=None if kw["q_weight"] is None else kw["q_weight"].cpu())
    u, tiny = util.half_step(dtype)
    for got in (out, same):
        util.check(got, ref, u * ref.abs() + 2.0 ** -20 * size + tiny, "q")


# ---------------------------------------------------------------- attention

DECODE = [
    ("f16", 2, 4, 64, 1, [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], {}),
    ("bf16", 8, 32, 128, 15, [5, 500, 0, 1000], {}),
    ("f16", 4, 4, 128, 3, [700, 20], dict(window=64)),
    ("bf16", 1, 8, 96, 7, [40, 513, 90], dict(window=33, prefix=[5, 0, 90])),
    ("f16", 2, 32, 80, 2, [129, 400], dict(cap=20.0)),
    ("bf16", 2, 2, 256, 1, [64, 257], dict(slopes=True)),
    ("f16", 1, 20, 192, 4, [77, 300], dict(cap=300.0, slopes=True)),
    ("bf16", 3, 3, 40, 5, [260, 13], dict(window=100, cap=30.0, slopes=True, prefix=[300, 2])),
    ("f16", 2, 2, 8, 1, [70], {}),
    ("bf16", 2, 2, 32, 1, [70, 200], {}),
    ("f16", 1, 16, 160, 1, [70, 200], {}),
    ("bf16", 1, 17, 224, 1, [70, 200], {}),
    ("f16", 4, 8, 128, 16, [3000], {}),
    ("f16", 40, 40, 128, 3, [90, 200, 1, 0, 33], {}),
    ("bf16", 64, 64, 64, 2, [90, 130], {}),
    ("f16", 15, 15, 96, 2, [70, 40], dict(slopes=True)),
    ("bf16", 10, 30, 128, 4, [290, 65], {}),
    ("f16", 6, 6, 200, 1, [150, 31], dict(cap=30.0)),
    ("bf16", 30, 30, 192, 1, [45, 130], {}),
    ("f16", 60, 60, 128, 1, [45, 130, 7], {}),
    ("bf16", 3, 3, 128, 8, list(range(0, 140)), {}),
]


def options(kw, hq, n):
    kw = dict(kw)
    slopes = torch.linspace(0.01, 0.5, hq) if kw.pop("slopes", False) else None
    prefix = kw.pop("prefix", None)
    cap = kw.pop("cap", 0.0)
    window = kw.pop("window", 0)
    ref = dict(cap=cap, window=window, slopes=slopes, prefix=prefix)
    own = dict(softcap=cap, window=window, slopes=None if slopes is None else slopes.cuda(),
               prefix_len=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"))
    return ref, own


def long_table(hk, n, tpp):
    """Blocks that make a table whose requests may have enough keys for the kernel of many keys."""
    return -(-2600000 // (hk * n * tpp))


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype,hk,hq,d,tpp,lens,kw", DECODE)
def test_decode(dtype, hk, hq, d, tpp, lens, kw, many):
    rng = np.random.default_rng(d + tpp)
    kw = dict(kw)
    if many and kw.get("window"):
        kw["window"] = 0  # (a window is few keys)
    c = four.Cache(rng, lens, dtype=dtype, hk=hk, d=d, tpp=tpp,
                   blocks_more=long_table(hk, len(lens), tpp) if many else 1)
    q = (torch.from_numpy(rng.standard_normal((len(lens), hq, d))) * 1.5).to(util.TORCH[dtype])
    ref_kw, own_kw = options(kw, hq, len(lens))
    scale = d ** -0.5
    cache, kt, vt = c.to_gpu()
    out = torch.full((len(lens), hq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros(len(lens), hq, device="cuda")
    cache.decode(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), lse=lse, **own_kw)
    ref = four.attention(c, q, [(r, n - 1) for r, n in enumerate(lens)], scale=scale, **ref_kw)
    worst = util.check(out, ref.out, four.bound(ref, dtype, True), "decode")
    print(f"[margin] {worst:.3f}")
    fine = torch.isfinite(ref.lse)
    assert torch.equal(torch.isneginf(lse.cpu()), ~fine)
    assert float((lse.cpu().double() - ref.lse)[fine].abs().max()) <= float(2 * ref.d.max()) + 1e-5


PREFILL = [
    ("f16", 2, 4, 64, 1, [0, 3, 100], [1, 17, 40], {}),
    ("bf16", 2, 8, 128, 15, [0, 130, 0], [70, 33, 0], {}),
    ("f16", 1, 3, 96, 7, [50, 0], [130, 1], dict(window=20)),
    ("bf16", 2, 2, 256, 2, [64, 5], [66, 9], dict(cap=25.0)),
    ("f16", 1, 4, 192, 1, [10, 200], [40, 3], dict(slopes=True)),
    ("bf16", 2, 2, 80, 3, [90, 400], [64, 2], dict(window=50, prefix=[7, 300])),
    ("f16", 2, 2, 40, 5, [1, 60], [65, 70], dict(cap=400.0)),
    ("bf16", 1, 5, 32, 4, [40, 10], [31, 33], dict(cap=30.0, slopes=True)),
    ("f16", 1, 1, 8, 1, [40], [31], {}),
    ("bf16", 1, 2, 160, 1, [40], [50], {}),
    ("f16", 1, 2, 224, 1, [40], [50], {}),
    ("bf16", 1, 4, 128, 4, [1500], [20], {}),
    ("f16", 1, 16, 72, 4, [900, 20], [5, 11], {}),
    ("bf16", 1, 64, 128, 15, [100], [70], {}),  # (read back first, and the next two)
    ("f16", 1, 64, 96, 4, [30, 0, 90], [70, 80, 60], dict(window=40, prefix=[9, 0, 70])),
    ("bf16", 1, 128, 80, 1, [0, 5], [33, 40], dict(cap=30.0, slopes=True)),
]


@pytest.mark.parametrize("dtype,hk,hq,d,tpp,past,new,kw", PREFILL)
def test_prefill(dtype, hk, hq, d, tpp, past, new, kw):
    rng = np.random.default_rng(d + tpp)
    lens = [a + b for a, b in zip(past, new)]
    c = four.Cache(rng, lens, dtype=dtype, hk=hk, d=d, tpp=tpp)
    T = sum(new)
    q = (torch.from_numpy(rng.standard_normal((T + 3, hq, d))) * 1.5).to(util.TORCH[dtype])
    ref_kw, own_kw = options(kw, hq, len(lens))
    cache, kt, vt = c.to_gpu()
    out = torch.full((T + 3, hq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros(T + 3, hq, device="cuda")
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets, lse=lse, **own_kw)
    rows = [(r, a + i) for r, (a, b) in enumerate(zip(past, new)) for i in range(b)]
    ref = four.attention(c, q[:T], rows, scale=d ** -0.5, **ref_kw)
    worst = util.check(out[:T], ref.out, four.bound(ref, dtype, False, back=T * hq // hk >= 4096 * len(lens)), "prefill")
    print(f"[margin] {worst:.3f}")
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 0).all())
    assert float((lse[:T].cpu().double() - ref.lse).abs().max()) <= float(2 * ref.d.max()) + 1e-5
