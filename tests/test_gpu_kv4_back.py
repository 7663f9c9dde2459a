"""Long prompts over the cache in 4 bits, whose keys are read back to 16 bits first: weights rounded to
the storage type once (2^-11 of a weight in f16, 2^-8 in bf16, as slora.h states for them; 64-bit
references and bounds of kv4_util), heads of every size, and what rows must not see."""

import math

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util

COUNT = 96     # keys of each of the two classes
MODES = {"plain": {}, "cap": dict(cap=20.0), "bias": dict(slopes=True), "cap and bias": dict(cap=20.0, slopes=True),
         "wide cap": dict(cap=400.0)}
TYPES = ["bf16", "f16"]


def rows_for(d):
    """Rows a request needs for its keys to be read back."""
    return 32 * d if d > 128 else 4096


def rounded_off(cap):
    """A scale and two levels below 6 whose weights, relative to the one of level 6, a rounding to bf16
    moves up and down by nearly 2^-8 of themselves."""
    levels = [4.0, 3.0, 2.0, 1.5, 1.0, 0.5, 0.0]
    scale = torch.arange(0.2, 0.9, 0.0002, dtype=torch.float64)
    s = [scale * x if not cap else cap * torch.tanh(scale * x / cap) for x in [6.0] + levels]
    w = [torch.exp(x - s[0]) for x in s[1:]]
    off = torch.stack([x.to(torch.bfloat16).double() / x - 1 for x in w])
    up, down = off.max(0), off.min(0)
    best = int((up.values - down.values).argmax())
    return float(scale[best].float()), levels[int(up.indices[best])], levels[int(down.indices[best])]


def weights_case(dtype, d, mode):
    """One level-6 key, two classes of COUNT keys whose values nearly cancel, new tokens that hardly
    weigh: what is left of the result is the weights' rounding."""
    kw = MODES[mode]
    scale, up, down = rounded_off(kw.get("cap", 0.0))
    hq = rows_for(d) // 32
    past, new = 1 + 2 * COUNT, 32
    c = four.Cache(np.random.default_rng(d), [past + new], dtype=dtype, hk=1, d=d, tpp=3)
    level = torch.cat([torch.tensor([6.0]), torch.full((COUNT,), up), torch.full((COUNT,), down), torch.full((new,), -6.0)]).double()
    k = torch.zeros(past + new, 1, d, dtype=torch.float64)
    k[:, 0, 0], k[:, 0, 1] = level, 6.0  # (step 1)
    cap = kw.get("cap", 0.0)
    s = scale * level if not cap else cap * torch.tanh(scale * level / cap)
    w = torch.exp(s - s[0])
    v = torch.zeros(past + new, 1, d, dtype=torch.float64)
    v[1:1 + COUNT] = 1.0
    v[1 + COUNT:past] = -float(w[1] / w[1 + COUNT])
    c.put(0, slice(0, past + new), 0, k)
    c.put(0, slice(0, past + new), 1, v)
    q = torch.zeros(new, hq, d)
    q[:, :, 0] = 1.0
    options = dict(cap=cap, slopes=torch.zeros(hq) if kw.get("slopes") else None)
    return c, q.to(util.TORCH[dtype]), [(0, past + i) for i in range(new)], scale, options


@pytest.mark.parametrize("mode", sorted(MODES))
def test_the_bounds_tell_the_types_apart(mode):
    """Weights rounded to bf16 are outside f16's bound, and near bf16's but inside."""
    c, q, rows, scale, options = weights_case("bf16", 64, mode)
    q = q[:, :1]
    if options["slopes"] is not None:
        options["slopes"] = options["slopes"][:1]
    good = four.attention(c, q, rows, scale=scale, **options)
    bad = four.attention(c, q, rows, scale=scale, rounded=torch.bfloat16, **options)
    f16 = four.attention(c, q, rows, scale=scale, rounded=torch.float16, **options)
    assert bool(((bad.out - good.out).abs() > 2 * four.bound(good, "f16", False, back=True)).all())
    assert bool(((f16.out - good.out).abs() <= four.bound(good, "f16", False, back=True)).all())
    bound = four.bound(good, "bf16", False, back=True)
    assert bool(((bad.out - good.out).abs() > bound / 2).all()) and bool(((bad.out - good.out).abs() <= bound).all())


@pytest.mark.gpu
@pytest.mark.parametrize("mode", sorted(MODES))
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 96), ("bf16", 128), ("bf16", 192), ("bf16", 256), ("f16", 128)])
def test_weights(dtype, d, mode):
    c, q, rows, scale, options = weights_case(dtype, d, mode)
    cache, kt, vt = c.to_gpu()
    out = torch.full_like(q, 7.0, device="cuda")
    slopes = options["slopes"]
    cache.prefill(q.cuda(), out, kt, vt, torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                  torch.tensor([0, len(rows)], dtype=torch.int32, device="cuda"), scale=scale, softcap=options["cap"],
                  slopes=None if slopes is None else slopes.cuda())
    ref = four.attention(c, q, rows, scale=scale, **options)
    worst = util.check(out, ref.out, four.bound(ref, dtype, False, back=True), "weights")
    print(f"[margin] {worst:.3f}")


CASES = [
    (160, 2, 3, [0, 90], [45, 36], {}),
    (192, 1, 1, [7], [50], dict(cap=30.0)),
    (224, 1, 4, [200], [60], dict(window=40, prefix=[9])),
    (256, 1, 2, [5, 0], [70, 62], dict(slopes=True)),
    (256, 2, 15, [64], [65], dict(cap=300.0, window=50)),
    (200, 1, 7, [260], [52], dict(cap=30.0, slopes=True, prefix=[33], window=100)),
    (128, 1, 15, [350], [70], {}),
    (40, 3, 2, [3, 70, 0], [40, 70, 33], dict(window=20, prefix=[0, 80, 5])),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,hk,tpp,past,new,kw", CASES)
def test_heads_masks_and_values_not_seen(dtype, d, hk, tpp, past, new, kw):
    """Keys of the last request that no row's window holds are NaN, in K and V; so is the V of a key that
    two rows see."""
    rng = np.random.default_rng(d + hk)
    lens = [a + b for a, b in zip(past, new)]
    group = -(-rows_for(d) * len(lens) // sum(new))
    hq = hk * group
    c = four.Cache(rng, lens, dtype=dtype, hk=hk, d=d, tpp=tpp)
    nan = torch.full((1, hk, d), math.nan, dtype=torch.float64)
    c.put(0, slice(lens[0] - 2, lens[0] - 1), 1, nan)  # the last two rows see it
    window, prefix = kw.get("window", 0), kw.get("prefix")
    if window:
        first = max(past[-1] - window + 1, 0)  # the first new row's first key
        for j in range(max(first - 5, 0 if prefix is None else prefix[-1]), first):
            for which in range(2):
                c.put(len(lens) - 1, slice(j, j + 1), which, nan)
    T = sum(new)
    q = (torch.from_numpy(rng.standard_normal((T + 2, hq, d))) * 1.5).to(util.TORCH[dtype])
    slopes = torch.linspace(0.01, 0.5, hq) if kw.get("slopes") else None
    cache, kt, vt = c.to_gpu()
    out = torch.full((T + 2, hq, d), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.zeros(T + 2, hq, device="cuda")
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, torch.tensor(lens, dtype=torch.int32, device="cuda"), offsets, lse=lse,
                  softcap=kw.get("cap", 0.0), window=window, slopes=None if slopes is None else slopes.cuda(),
                  prefix_len=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"))
    rows = [(r, a + i) for r, (a, b) in enumerate(zip(past, new)) for i in range(b)]
    ref = four.attention(c, q[:T], rows, scale=d ** -0.5, cap=kw.get("cap", 0.0), window=window, slopes=slopes, prefix=prefix)
    worst = util.check(out[:T], ref.out, four.bound(ref, dtype, False, back=True), "prefill")
    print(f"[margin] {worst:.3f}")
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 0).all())
    assert float((lse[:T].cpu().double() - ref.lse).abs().max()) <= float(2 * ref.d.max()) + 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 192), ("f16", 128)])
def test_wide_tables_are_read_straight(dtype, d):
    """The same prompt in a table with room for more than 4 keys a row: no workspace for them, and the
    weights' rounding is that of the other way."""
    c, q, rows, scale, _ = weights_case(dtype, d, "plain")
    wide = 4 * rows_for(d) // c.tpp + 64
    cache, _, _ = c.to_gpu()
    tables = [torch.from_numpy(np.pad(t, ((0, 0), (0, wide - t.shape[1])), constant_values=-1)).cuda() for t in (c.kt, c.vt)]
    from heterogeneous_lora_amd import _lib
    a = _lib.Attn(n_q_heads=q.shape[1])
    of_16_bits = _lib.KV(1 << 20, 1, c.tpp * d, _lib.DTYPES[dtype], 1, d, c.tpp, 1, wide)
    assert cache.workspace_size(cache._kv(1, wide), a, len(rows)) == _lib.attn_workspace_size(of_16_bits, a, len(rows))
    out = torch.full_like(q, 7.0, device="cuda")
    cache.prefill(q.cuda(), out, *tables, torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                  torch.tensor([0, len(rows)], dtype=torch.int32, device="cuda"), scale=scale)
    ref = four.attention(c, q, rows, scale=scale)
    util.check(out, ref.out, four.bound(ref, dtype, False), "straight")
