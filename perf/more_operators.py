"""A KV cache held in 4 bits: the cases that are measured, and their plain forms.

Four operators of a serving step whose cache takes 4.25 bits a value (heads of 128) in the unified pool's pages.
32 neighbouring dimensions of a head's vector share a step; a value is its step times one of
0, 0.5, 1, 1.5, 2, 3, 4, 6 or their negatives. `_layout` says how a token lies in a page.

* write: per-head norm of q and k, rotary positions, q in 16 bits, K and V quantised to their slots, and what the
  cache then holds read back (as a step does that hands new keys on to a 16-bit path).
* read: the K and V of tokens anywhere in the pool, in 16 bits.
* decode: attention of one new token per request over its cached keys.
* prefill: attention of the new tokens of each request (its last ones) over its cached keys: causal, with an optional
  sliding window, prefix, score cap and distance bias.

`run` computes them with elementary torch operations where `own` is False, and calls the library's entry points where
it is True.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the smallest call: one token of a small layer
        dict(name="write_one", op="write", dtype="f16", tokens=1, q_heads=4, kv_heads=4, dim=64, rotary=64,
             interleaved=False, norm=False, scaling="none", factor=1.0, tpp=1, page_elems=256, pos_hi=512),
        # a decode batch of 256 tokens, width 4096
        dict(name="write_decode", op="write", dtype="f16", tokens=256, q_heads=32, kv_heads=32, dim=128, rotary=128,
             interleaved=False, norm=False, scaling="none", factor=1.0, tpp=3, page_elems=4096, pos_hi=2048),
        # prompts of 16411 tokens in all, shared key heads, norms, half of each head rotated, long positions
        dict(name="write_prefill", op="write", dtype="bf16", tokens=16411, q_heads=32, kv_heads=8, dim=128, rotary=64,
             interleaved=True, norm=True, scaling="bands", factor=8.0, tpp=15, page_elems=4096, pos_hi=1000000),
        # the newest tokens of 17 requests, heads of an odd size
        dict(name="read_few", op="read", dtype="f16", tokens=17, kv_heads=8, dim=80, tpp=7, page_elems=4096),
        # a long prefix handed to a 16-bit path
        dict(name="read_prefix", op="read", dtype="bf16", tokens=65000, kv_heads=8, dim=128, tpp=15, page_elems=4096),
        # the smallest call: one short request
        dict(name="decode_one", op="decode", dtype="f16", requests=1, q_heads=32, kv_heads=32, dim=128,
             len_lo=33, len_hi=33, tpp=3, page_elems=4096, window=0, prefix=0, cap=0.0, slopes=False),
        # the decode half of a mixed batch, width 5120: 512 requests, 64 to 2048 tokens cached
        dict(name="decode_mixed", op="decode", dtype="f16", requests=512, q_heads=40, kv_heads=40, dim=128,
             len_lo=64, len_hi=2048, tpp=3, page_elems=5120, window=0, prefix=0, cap=0.0, slopes=False),
        # few requests with long caches, 8 query heads to a key head
        dict(name="decode_long", op="decode", dtype="bf16", requests=3, q_heads=64, kv_heads=8, dim=128,
             len_lo=100000, len_hi=131072, tpp=15, page_elems=4096, window=0, prefix=0, cap=0.0, slopes=False),
        # window, kept prefix, cap and distance bias together, an odd head size
        dict(name="decode_window", op="decode", dtype="bf16", requests=64, q_heads=32, kv_heads=8, dim=96,
             len_lo=1, len_hi=8192, tpp=13, page_elems=4096, window=1024, prefix=16, cap=30.0, slopes=True),
        # the smallest call: two short prompts
        dict(name="prefill_small", op="prefill", dtype="f16", requests=2, q_heads=4, kv_heads=4, dim=64,
             past_lo=0, past_hi=0, new_lo=1, new_hi=17, tpp=3, page_elems=256, window=0, prefix=0,
             cap=0.0, slopes=False),
        # 64 prompts of 8 to 512 tokens, width 4096
        dict(name="prefill_batch", op="prefill", dtype="bf16", requests=64, q_heads=32, kv_heads=32, dim=128,
             past_lo=0, past_hi=0, new_lo=8, new_hi=512, tpp=3, page_elems=4096, window=0, prefix=0,
             cap=0.0, slopes=False),
        # two long prompts continued after cached parts, 4 query heads to a key head
        dict(name="prefill_long", op="prefill", dtype="bf16", requests=2, q_heads=32, kv_heads=8, dim=128,
             past_lo=7000, past_hi=8192, new_lo=8000, new_hi=8192, tpp=15, page_elems=4096, window=0, prefix=0,
             cap=0.0, slopes=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "prefill"])
    kv_heads = rng.choice([1, 2, 4, 8, 5, 10, 32])
    dim = rng.choice([64, 128, 128, 80, 96, 256])
    tpp = rng.choice([1, 2, 3, 4, 7, 15])
    heads = dict(dtype=rng.choice(["bf16", "f16"]), kv_heads=kv_heads, dim=dim, tpp=tpp)
    heads["page_elems"] = _ceil(tpp * _layout(heads)[2], 16) * 8 + rng.choice([0, 0, 8, 64])
    if op == "read":
        return dict(op=op, tokens=min(_log_int(rng, 1, 65000), 65000 * 8 * 128 // (kv_heads * dim)), **heads)
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    if kv_heads * group > 64:
        group = 1
    heads["q_heads"] = kv_heads * group
    if op == "write":
        tokens = min(_log_int(rng, 1, 16384), 16411 * 48 * 128 // (kv_heads * (group + 2) * dim))
        return dict(op=op, tokens=tokens, rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), pos_hi=_log_int(rng, 64, 1000000), **heads)
    options = dict(window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), prefix=rng.choice([0, 0, _log_int(rng, 1, 512)]),
                   cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3)
    if op == "decode":
        requests = _log_int(rng, 1, 512)
        most = min(131072, max(1, int(1e9 / (requests * kv_heads * dim))))
        len_hi = _log_int(rng, 1, most)
        return dict(op=op, requests=requests, len_lo=rng.randint(0, len_hi), len_hi=len_hi, **options, **heads)
    requests = _log_int(rng, 1, 64)
    most = max(1, min(8192, int(math.sqrt(1.5e9 / (requests * kv_heads * group)))))
    new_hi = _log_int(rng, 1, most)
    past_hi = rng.choice([0, _log_int(rng, 1, most)])
    return dict(op=op, requests=requests, past_lo=rng.randint(0, past_hi), past_hi=past_hi,
                new_lo=rng.randint(0, new_hi), new_hi=new_hi, **options, **heads)


# ---------------------------------------------------------------- the cache's layout

def _ceil(a, b):
    return -(-a // b)


def _layout(case):
    """Groups of 32 dimensions in a head, bytes of a head's steps, bytes of a token's K (or V) in a page.

    A token: the heads' codes, 16 bytes a group, then the heads' steps, a byte a group (padded to 1, 2, 4 or 8), the
    whole rounded up to 16 bytes. Code bytes go [dimension / 8 % 4][group][4 bytes], two dimensions a byte, the lower
    one in the low bits. A code is its level's number, 8 more if negative; a step is the upper 8 bits below the sign
    of its 16-bit float."""
    groups = _ceil(case["dim"], 32)
    steps = 1 if groups == 1 else 2 if groups == 2 else 4 if groups <= 4 else 8
    return groups, steps, _ceil(case["kv_heads"] * (16 * groups + steps), 16) * 16


def _grouped(case, x):
    """[n, kv heads, dim] -> [n, kv heads, groups, 32], zeros behind the head's end."""
    groups = _layout(case)[0]
    return torch.nn.functional.pad(x, (0, 32 * groups - case["dim"])).unflatten(-1, (groups, 32))


def _steps_of(x):
    """The steps of [..., 32] values: the largest magnitude / 6, rounded to 4 significant bits (2^-17 at least apart)."""
    most = x.abs().amax(-1) / 6
    apart = torch.exp2(torch.frexp(most)[1].clamp(min=-13) - 4.0).to(x.dtype)
    return (torch.round(most / apart) * apart).clamp(max=10240.0)


def _codes_of(x, step):
    """The nearest level's number (the even one of two equally near), 8 more where negative."""
    t = x.abs() / torch.where(step == 0, 1.0, step)[..., None]
    n = torch.where(t < 2, torch.round(2 * t), torch.where(t < 4, torch.round(t) + 2, torch.round(t / 2) + 4))
    return n.clamp(max=7).to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)


def _values(codes, step):
    levels = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=step.dtype, device=step.device)
    return levels[codes.int()] * step[..., None]


def _token_bytes(case, x):
    """Tokens [n, kv heads, dim] as they lie in a page, [n, bytes]."""
    groups, steps, size = _layout(case)
    x = _grouped(case, x)
    step = _steps_of(x)
    code = _codes_of(x, step).unflatten(-1, (4, 4, 2))  # [n, heads, group, dimension / 8 % 4, byte, half]
    code = (code[..., 0] | code[..., 1] << 4).transpose(2, 3).flatten(1)
    row = torch.zeros(x.shape[0], size, dtype=torch.uint8, device=x.device)
    row[:, :code.shape[1]] = code
    byte = (step.half().view(torch.int16) >> 7).to(torch.uint8)
    row[:, code.shape[1]:code.shape[1] + case["kv_heads"] * steps] = \
        torch.nn.functional.pad(byte, (0, steps - groups)).flatten(1)
    return row


def _rows(s, page, inside):
    """The tokens' bytes, of page `page` and place `inside` in it."""
    case, size = s["case"], _layout(s["case"])[2]
    pages = s["pool"].view(torch.uint8).view(s["n_pages"], -1)
    return pages[:, :case["tpp"] * size].unflatten(1, (case["tpp"], size))[page, inside]


def _dequantised(case, row):
    """[..., bytes] -> [..., kv heads, dim] in 32 bits."""
    groups, steps, _ = _layout(case)
    hk, d = case["kv_heads"], case["dim"]
    pairs = torch.tensor([[a, b] for b in LEVELS + tuple(-x for x in LEVELS) for a in LEVELS + tuple(-x for x in LEVELS)],
                         device=row.device)
    n = hk * 16 * groups
    x = torch.nn.functional.embedding(row[..., :n].int(), pairs).view(*row.shape[:-1], hk, 4, groups, 8)
    byte = row[..., n:n + hk * steps].unflatten(-1, (hk, steps))[..., :groups]
    step = (byte.to(torch.int16) << 7).view(torch.float16).float()
    x = (x * step[..., None, :, None]).transpose(-3, -2)
    return x.reshape(*row.shape[:-1], hk, 32 * groups)[..., :d]


# ---------------------------------------------------------------- inputs

def _lengths(case, seed, lo, hi, salt):
    """Lengths spread evenly from lo to hi, in an order of the seed's (a batch's size is the case's own)."""
    n, a, b = case["requests"], case[lo], case[hi]
    spread = [b if n == 1 else a + (b - a) * i // (n - 1) for i in range(n)]
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed * 8 + salt)).tolist()
    return [spread[i] for i in order]


def _rope_turns(case):
    """Turns per position of each rotated pair (float64), and the factor on cos and sin (a 32-bit number)."""
    d, theta, f = case["rotary"], 10000.0, case["factor"]
    if case["scaling"] == "base":
        theta = theta * f ** (d / (d - 2))
    t = theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) / (2 * math.pi)
    if case["scaling"] == "linear":
        t = t / f
    if case["scaling"] == "bands":  # slow pairs are stretched, fast ones kept, a linear blend between
        keep = ((t * 8192 - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        t = t * keep + t / f * (1.0 - keep)
        return t, float(torch.tensor(0.1 * math.log(f) + 1.0, dtype=torch.float32))
    return t, 1.0


def _pool(case, n_pages, g):
    """A pool whose every place holds a token: K as after a norm, V of the same scale."""
    dev, hk, d, tpp = "cuda", case["kv_heads"], case["dim"], case["tpp"]
    size = _layout(case)[2]
    pool = torch.zeros(n_pages, 2 * case["page_elems"], dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (tpp * hk * d))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        pool[i:i + n, :tpp * size] = _token_bytes(case, torch.randn(n * tpp, hk, d, generator=g, device=dev)).view(n, -1)
    return pool.view(torch.int16).flatten()


def _cache(case, lens, g):
    """A pool that holds `lens` tokens' K and V on shuffled pages, and the two block tables."""
    dev, tpp = "cuda", case["tpp"]
    blocks = [_ceil(n, tpp) for n in lens]
    most = max(max(blocks), 1)
    n_pages = 2 * sum(blocks) + 3
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    inside = torch.arange(most, device=dev)[None, :] < torch.tensor(blocks, device=dev)[:, None]
    tables = []
    for part in range(2):
        t = torch.full((len(lens), most), -1, dtype=torch.int32, device=dev)
        t[inside] = ids[part * sum(blocks):(part + 1) * sum(blocks)]
        tables.append(t)
    return _pool(case, n_pages, g), n_pages, tables[0], tables[1]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    kind, d, hk = TYPES[case["dtype"]], case["dim"], case["kv_heads"]
    if case["op"] in ("write", "read"):
        t = case["tokens"]
        each = _ceil(t, case["tpp"]) + 2
        order = torch.randperm(2 * each, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        k_slots, v_slots = (order[i * each:][at // case["tpp"]] * case["tpp"] + at % case["tpp"] for i in range(2))
        s.update(n_pages=2 * each, pool=_pool(case, 2 * each, g), k_slots=k_slots, v_slots=v_slots,
                 k_out=torch.zeros(t, hk, d, dtype=kind, device=dev), v_out=torch.zeros(t, hk, d, dtype=kind, device=dev))
        if case["op"] == "write":
            hq = case["q_heads"]
            packed = torch.randn(t, (hq + 2 * hk) * d, generator=g, device=dev).to(kind)  # one projection's rows
            q, k, v = (x.view(t, -1, d) for x in packed.split([hq * d, hk * d, hk * d], dim=1))
            turns, factor = _rope_turns(case)
            s.update(q=q, k=k, v=v, q_out=torch.zeros(t, hq, d, dtype=kind, device=dev), turns=turns.to(dev),
                     position=torch.randint(0, case["pos_hi"], (t,), generator=g, device=dev, dtype=torch.int32),
                     factor=factor, q_weight=None, k_weight=None)
            if case["norm"]:
                s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(kind)
                s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(kind)
    else:
        hq = case["q_heads"]
        if case["op"] == "decode":
            new = [1] * case["requests"]
            lens = _lengths(case, seed, "len_lo", "len_hi", 1)
        else:
            new = _lengths(case, seed, "new_lo", "new_hi", 2)
            lens = [a + b for a, b in zip(_lengths(case, seed, "past_lo", "past_hi", 1), new)]
        pool, n_pages, kt, vt = _cache(case, lens, g)
        q = torch.randn(sum(new), hq, d, generator=g, device=dev) * 1.5
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        s.update(pool=pool, n_pages=n_pages, k_table=kt, v_table=vt, lens=lens, offsets=offsets, q=q.to(kind),
                 out=torch.zeros(sum(new), hq, d, dtype=kind, device=dev), scale=1.0 / math.sqrt(d),
                 seq_len=torch.tensor(lens, dtype=torch.int32, device=dev),
                 q_offsets=torch.tensor(offsets, dtype=torch.int32, device=dev), slopes=None, prefix_len=None)
        if case["slopes"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=dev, dtype=torch.float32) / hq)
        if case["prefix"]:
            s["prefix_len"] = torch.full((case["requests"],), case["prefix"], dtype=torch.int32, device=dev)
    if own:
        s["calls"] = _bind(s)
    return s


def _bind(s):
    """The library's calls on this state, their arguments marshalled once, as a serving loop keeps them."""
    from heterogeneous_lora_amd import runtime
    case = s["case"]
    cache = runtime.KVCache(s["pool"], s["n_pages"], page_elems=case["page_elems"], dtype=case["dtype"],
                            n_kv_heads=case["kv_heads"], head_dim=case["dim"], tokens_per_page=case["tpp"], bits=4)
    if case["op"] in ("write", "read"):
        read = cache.bind_read(s["k_out"], s["v_out"], s["k_slots"], s["v_slots"])
        if case["op"] == "read":
            return [read]
        rope = runtime.Rope(case["rotary"], theta=10000.0, interleaved=case["interleaved"], scaling=case["scaling"],
                            factor=case["factor"], original_len=8192, low_turns=1.0, high_turns=4.0,
                            cos_sin_scale=s["factor"])
        return [cache.bind_write(s["q"], s["k"], s["v"], s["q_out"], s["position"], s["k_slots"], s["v_slots"],
                                 rope=rope, norm=case["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 eps=2.0 ** -20), read]
    options = dict(scale=s["scale"], softcap=case["cap"], window=case["window"], slopes=s["slopes"],
                   prefix_len=s["prefix_len"])
    if case["op"] == "decode":
        return [cache.bind_decode(s["q"], s["out"], s["k_table"], s["v_table"], s["seq_len"], **options)]
    return [cache.bind_prefill(s["q"], s["out"], s["k_table"], s["v_table"], s["seq_len"], s["q_offsets"], **options)]


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        for call in s["calls"]:
            call()
        if op == "read":
            return dict(k=s["k_out"], v=s["v_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"]) if op == "write" else s["out"]
    return _plain_write(s) if op == "write" else _plain_read(s) if op == "read" else _plain_attention(s)


def _plain_write(s):
    case, r, kind = s["case"], s["case"]["rotary"], s["q"].dtype
    angle = s["position"].double()[:, None] * s["turns"][None, :]
    angle = (angle - angle.floor()) * (2 * math.pi)
    cos, sin = (angle.cos() * s["factor"])[:, None, :], (angle.sin() * s["factor"])[:, None, :]

    def turned(x, weight, wide):
        x, c, n = x.to(wide), cos.to(wide), sin.to(wide)
        if case["norm"]:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 2.0 ** -20) * weight.to(wide)
        rot, rest = x[..., :r], x[..., r:]
        if case["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
        else:
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            rot = torch.cat([a * c - b * n, b * c + a * n], -1)
        return torch.cat([rot, rest], -1)

    def held(x):
        x = _grouped(case, x)
        step = _steps_of(x)
        return _values(_codes_of(x, step), step).flatten(-2)[..., :case["dim"]].to(kind)

    # (K next to a border between two levels: in 64 bits)
    return dict(q=turned(s["q"], s["q_weight"], torch.float32).to(kind),
                k=held(turned(s["k"], s["k_weight"], torch.float64)), v=held(s["v"].double()))


def _plain_read(s):
    case, kind = s["case"], s["k_out"].dtype
    k, v = (_dequantised(case, _rows(s, at // case["tpp"], at % case["tpp"])).to(kind)
            for at in (s["k_slots"], s["v_slots"]))
    return dict(k=k, v=v)


def _plain_attention(s):
    """All requests together, padded to the longest, a few key heads at a time."""
    case, out = s["case"], s["out"]
    hk, group, d, tpp = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["dim"], case["tpp"]
    dev = out.device
    most = max(max(s["lens"]), 1)
    begin, seq = s["q_offsets"][:-1].long(), s["seq_len"].long()
    new = s["q_offsets"].long().diff()
    rows = max(b - a for a, b in zip(s["offsets"], s["offsets"][1:]))
    if rows == 0:
        return out
    key, row = torch.arange(most, device=dev), torch.arange(rows, device=dev)
    pages = (t.long()[:, key // tpp].clamp(min=0) for t in (s["k_table"], s["v_table"]))
    k, v = (_dequantised(case, _rows(s, p, (key % tpp).expand_as(p))) for p in pages)  # [requests, keys, heads, dim]
    k, v = k.permute(0, 2, 3, 1).contiguous(), v.transpose(1, 2).contiguous()
    q = s["q"][(begin[:, None] + row).clamp(max=out.shape[0] - 1)].float().unflatten(2, (hk, group))
    pos = (seq - new)[:, None] + row  # [requests, rows]
    far = key - pos[:, :, None]
    seen = far <= 0
    if case["window"]:
        seen &= far > -case["window"]
    if case["prefix"]:
        seen |= key < case["prefix"]
    seen = (seen & (key < seq[:, None, None]))[:, None, None]
    y = torch.empty(len(seq), hk, group * rows, d, device=dev)
    few = max(1, int(3e9) // max(1, group * rows * most * len(seq)))
    for h in range(0, hk, few):
        e = min(h + few, hk)
        x = q[:, :, h:e].permute(0, 2, 3, 1, 4).reshape(len(seq), e - h, group * rows, d)
        x = torch.matmul(x, k[:, h:e]).unflatten(2, (group, rows)) * s["scale"]
        if case["cap"]:
            x = case["cap"] * torch.tanh(x / case["cap"])
        if case["slopes"]:
            x = x + s["slopes"].view(1, hk, group, 1, 1)[:, h:e] * far[:, None, None]
        x = torch.where(seen, x, -math.inf)
        x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=torch.finfo(x.dtype).min))
        x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
        y[:, h:e] = torch.matmul(x.flatten(2, 3), v[:, h:e])
    y = y.unflatten(2, (group, rows)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [requests, rows, query heads, dim]
    out.copy_(y[row < new[:, None]])
    return out


# ---------------------------------------------------------------- the work of one pass

def work(case):
    hq, hk, d = case.get("q_heads"), case["kv_heads"], case["dim"]
    held = hk * (d / 2 + _ceil(d, 32))  # bytes of a token's K
    if case["op"] == "read":
        return dict(bytes=case["tokens"] * (2 * held + 4 * hk * d + 16), flops=0)
    if case["op"] == "write":  # (and its values read back)
        t = case["tokens"]
        return dict(bytes=t * (4 * hq * d + 4 * hk * d + 2 * held + 20 + 2 * held + 4 * hk * d + 16),
                    flops=t * (hq + hk) * (3 * case["rotary"] + 4 * d))
    if case["op"] == "decode":
        lens, new = _lengths(case, 0, "len_lo", "len_hi", 1), [1] * case["requests"]
    else:
        new = _lengths(case, 0, "new_lo", "new_hi", 2)
        lens = [a + b for a, b in zip(_lengths(case, 0, "past_lo", "past_hi", 1), new)]
    w, pre = case["window"], case["prefix"]
    keys = pairs = 0
    for n, m in zip(lens, new):  # keys that some query sees, and seen pairs (a window cuts both)
        keys += min(n, w + m - 1 + pre) if w and m else n if m else 0
        pairs += min(m * (n - m) + m * (m + 1) // 2, m * (w + pre) if w else n * m)
    return dict(bytes=keys * 2 * held + 4 * sum(new) * hq * d + 4 * case["requests"], flops=4 * pairs * hq * d)


# ---------------------------------------------------------------- exact results

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    if case["op"] == "read":
        return dict(k=_exact_rows(s, s["k_slots"]), v=_exact_rows(s, s["v_slots"]))
    return _exact_attention(s)


def _step_table(device):
    """The steps of bytes 0 .. 226 (the largest whose 6-fold is a finite 16-bit float)."""
    b = torch.arange(227, device=device)
    e, m = (b >> 3).double(), (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, torch.exp2(e - 15) * (1 + m / 8))


def _exact_rows(s, slots):
    """The vectors at `slots`, dimension by dimension out of the pool's bytes, in 64 bits."""
    case = s["case"]
    hk, d, tpp = case["kv_heads"], case["dim"], case["tpp"]
    groups, steps, size = _layout(case)
    flat = s["pool"].view(torch.uint8)
    i = torch.arange(d, device=flat.device)
    h = torch.arange(hk, device=flat.device)[:, None]
    code_at = h * 16 * groups + (i // 8 % 4 * groups + i // 32) * 4 + i % 8 // 2
    step_at = hk * 16 * groups + h * steps + i // 32
    base = (slots // tpp * (2 * case["page_elems"]) + slots % tpp * size)[:, None, None]
    code = flat[base + code_at] >> (i % 2 * 4).to(torch.uint8) & 15
    level = torch.tensor(LEVELS, dtype=torch.float64, device=flat.device)[(code & 7).long()]
    return torch.where(code >= 8, -level, level) * _step_table(flat.device)[flat[base + step_at].long()]


def _nearest(x, marks):
    """How many of the midpoints between rising `marks` lie below x; at one, the even number."""
    mids = (marks[1:] + marks[:-1]) / 2
    n = torch.searchsorted(mids, x.contiguous())
    tie = (n < len(mids)) & (mids[n.clamp(max=len(mids) - 1)] == x)
    return torch.where(tie & (n % 2 == 1), n + 1, n)


def _exact_held(case, x):
    """What the cache holds of x: a step and a level by their distances."""
    x = _grouped(case, x)
    steps = _step_table(x.device)
    step = steps[_nearest(x.abs().amax(-1), 6 * steps)][..., None]
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    size = level[_nearest(x.abs() / torch.where(step == 0, math.inf, step), level)] * step
    return torch.where(x < 0, -size, size).flatten(-2)[..., :case["dim"]]


def _exact_write(s):
    """Each rotated pair as a complex number times e^(2 pi i position turns)."""
    case, r = s["case"], s["case"]["rotary"]
    turns = torch.remainder(s["position"].double()[:, None] * s["turns"], 1.0)
    unit = torch.polar(torch.full_like(turns, s["factor"]), 2 * math.pi * turns)[:, None, :]
    result = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 2.0 ** -20) * weight.double()
        y = y.clone()
        if case["interleaved"]:
            first, second = y[..., 0:r:2], y[..., 1:r:2]
        else:
            first, second = y[..., 0:r // 2], y[..., r // 2:r]
        z = torch.complex(first.contiguous(), second.contiguous()) * unit
        first.copy_(z.real)
        second.copy_(z.imag)
        result.append(y)
    return dict(q=result[0], k=_exact_held(case, result[1]), v=_exact_held(case, s["v"].double()))


def _exact_attention(s):
    """Request by request, head by head and in blocks of queries, in 64 bits."""
    case = s["case"]
    if work(case)["flops"] > 2e13:
        return None
    hk, d, tpp = case["kv_heads"], case["dim"], case["tpp"]
    group = case["q_heads"] // hk
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for r, n in enumerate(s["lens"]):
        a, b = s["offsets"][r], s["offsets"][r + 1]
        if n == 0 or a == b:
            continue
        j = torch.arange(n, device=out.device)
        if case["op"] == "decode" and case["window"]:  # only keys that are seen
            j = j[(j >= n - case["window"]) | (j < case["prefix"])]
        k, v = (_exact_rows(s, t[r].long()[j // tpp] * tpp + j % tpp) for t in (s["k_table"], s["v_table"]))
        for c in range(a, b, 1024):
            e = min(c + 1024, b)
            i = torch.arange(n - (b - c), n - (b - e), device=out.device)
            far = (i[:, None] - j[None, :])
            keep = far >= 0
            if case["window"]:
                keep = keep & (far < case["window"])
            if case["prefix"]:
                keep = keep | (j < case["prefix"])[None, :]
            keep = keep.repeat_interleave(group, 0)
            for h in range(hk):
                x = s["q"][c:e, h * group:(h + 1) * group].double().reshape(-1, d)
                score = torch.mm(x, k[:, h].t().contiguous()) * s["scale"]
                if case["cap"]:
                    score = torch.tanh(score / case["cap"]) * case["cap"]
                if case["slopes"]:
                    slope = s["slopes"][h * group:(h + 1) * group].double().repeat(e - c)
                    score = score - slope[:, None] * far.repeat_interleave(group, 0)
                score = score.masked_fill(~keep, -math.inf)
                y = torch.mm(torch.softmax(score, -1), v[:, h].contiguous())
                out[c:e, h * group:(h + 1) * group] = y.view(e - c, group, d)
    return out
