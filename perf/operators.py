"""Attention over the unified pool's KV pages: the cases that are measured, and their plain forms.

Four operators, used together in a serving step. Pages are those of the unified pool: one page
holds `tpp` tokens' K (or V) vectors of one layer, [tpp][kv heads][head dim], and a request's
tokens lie on pages anywhere in the pool.

* tables: from request lengths and the page ids in allocation order, the block table of every
  plane (a layer's K or V), the slot of every new token, positions, request ids and offsets.
* write: per-head norm of q and k, rotary positions, K and V stored to their slots, in one pass.
* decode: attention of one new token per request over its cached keys.
* prefill: attention of the new tokens of each request (its last ones) over its cached keys:
  causal, with an optional sliding window, prefix, score cap and distance bias.

`run` computes them with elementary torch operations where `own` is False, and calls the
library's entry points where it is True.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of a 32-layer model (64 planes), 256 running requests: one new block each
        dict(name="tables_step", op="tables", requests=256, planes=64, tpp=1, append=True,
             past_lo=64, past_hi=2048, new_lo=1, new_hi=1, max_blocks=2176),
        # the whole tables of 560 sequences of a 40-layer model, after requests were reordered
        dict(name="tables_rebuild", op="tables", requests=560, planes=80, tpp=1, append=False,
             past_lo=64, past_hi=2048, new_lo=0, new_hi=256, max_blocks=2304),
        # the smallest call: one token of a small layer
        dict(name="write_one", op="write", dtype="f16", tokens=1, q_heads=4, kv_heads=4, dim=64,
             rotary=64, interleaved=False, norm=False, scaling="none", factor=1.0, tpp=1,
             page_elems=256, pos_hi=512),
        # a decode batch of 256 tokens, width 4096
        dict(name="write_decode", op="write", dtype="f16", tokens=256, q_heads=32, kv_heads=32, dim=128,
             rotary=128, interleaved=False, norm=False, scaling="none", factor=1.0, tpp=1,
             page_elems=4096, pos_hi=2048),
        # prompts of 16411 tokens in all, shared key heads, norms, half of each head rotated, long positions
        dict(name="write_prefill", op="write", dtype="bf16", tokens=16411, q_heads=32, kv_heads=8, dim=128,
             rotary=64, interleaved=True, norm=True, scaling="bands", factor=8.0, tpp=4,
             page_elems=4096, pos_hi=1000000),
        # the smallest call: one short request
        dict(name="decode_one", op="decode", dtype="f16", requests=1, q_heads=32, kv_heads=32, dim=128,
             len_lo=33, len_hi=33, tpp=1, page_elems=4096, window=0, prefix=0, cap=0.0, slopes=False),
        # the decode half of a mixed batch, width 5120: 512 requests, 64 to 2048 tokens cached
        dict(name="decode_mixed", op="decode", dtype="f16", requests=512, q_heads=40, kv_heads=40, dim=128,
             len_lo=64, len_hi=2048, tpp=1, page_elems=5120, window=0, prefix=0, cap=0.0, slopes=False),
        # few requests with long caches, 8 query heads to a key head
        dict(name="decode_long", op="decode", dtype="bf16", requests=3, q_heads=64, kv_heads=8, dim=128,
             len_lo=100000, len_hi=131072, tpp=4, page_elems=4096, window=0, prefix=0, cap=0.0, slopes=False),
        # window, kept prefix, cap and distance bias together, an odd head size
        dict(name="decode_window", op="decode", dtype="bf16", requests=64, q_heads=32, kv_heads=8, dim=96,
             len_lo=1, len_hi=8192, tpp=5, page_elems=4096, window=1024, prefix=16, cap=30.0, slopes=True),
        # the smallest call: two short prompts
        dict(name="prefill_small", op="prefill", dtype="f16", requests=2, q_heads=4, kv_heads=4, dim=64,
             past_lo=0, past_hi=0, new_lo=1, new_hi=17, tpp=1, page_elems=256, window=0, prefix=0,
             cap=0.0, slopes=False),
        # 64 prompts of 8 to 512 tokens, width 4096
        dict(name="prefill_batch", op="prefill", dtype="bf16", requests=64, q_heads=32, kv_heads=32, dim=128,
             past_lo=0, past_hi=0, new_lo=8, new_hi=512, tpp=1, page_elems=4096, window=0, prefix=0,
             cap=0.0, slopes=False),
        # two long prompts continued after cached parts, 4 query heads to a key head, capped scores
        dict(name="prefill_long", op="prefill", dtype="bf16", requests=2, q_heads=32, kv_heads=8, dim=128,
             past_lo=7000, past_hi=8192, new_lo=8000, new_hi=8192, tpp=4, page_elems=4096, window=0, prefix=0,
             cap=50.0, slopes=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "decode", "prefill"])
    if op == "tables":
        requests = _log_int(rng, 1, 560)
        tpp = rng.choice([1, 1, 2, 3, 4, 16])
        past_hi = _log_int(rng, 1, 2000)
        new_hi = rng.choice([1, 1, _log_int(rng, 1, 256)])
        append = rng.random() < 0.5
        return dict(op=op, requests=requests, planes=2 * rng.randint(1, 40), tpp=tpp, append=append,
                    past_lo=rng.randint(0, past_hi), past_hi=past_hi, new_lo=rng.randint(0, 1), new_hi=new_hi,
                    max_blocks=-(-(past_hi + new_hi) // tpp) + rng.choice([0, 1, 37]))
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 80, 96, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 5, 10, 32])
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    if kv_heads * group > 64:
        group = 1
    tpp = rng.choice([1, 1, 2, 4, 7])
    heads = dict(dtype=dtype, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, tpp=tpp,
                 page_elems=tpp * kv_heads * dim + rng.choice([0, 0, 8, 64]))
    if op == "write":
        tokens = _log_int(rng, 1, 16384)
        if tokens * (kv_heads * (group + 2)) * dim > 16411 * 48 * 128:
            tokens = 16411 * 48 * 128 // (kv_heads * (group + 2) * dim)
        return dict(op=op, tokens=tokens, rotary=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), pos_hi=_log_int(rng, 64, 1000000), **heads)
    options = dict(window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), prefix=rng.choice([0, 0, _log_int(rng, 1, 512)]),
                   cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3)
    if op == "decode":
        requests = _log_int(rng, 1, 512)
        most = min(131072, max(1, int(5e8 / (requests * kv_heads * dim))))
        len_hi = _log_int(rng, 1, most)
        return dict(op=op, requests=requests, len_lo=rng.randint(0, len_hi), len_hi=len_hi, **options, **heads)
    requests = _log_int(rng, 1, 64)
    most = max(1, min(8192, int(math.sqrt(1.5e9 / (requests * kv_heads * group)))))
    new_hi = _log_int(rng, 1, most)
    past_hi = rng.choice([0, _log_int(rng, 1, most)])
    return dict(op=op, requests=requests, past_lo=rng.randint(0, past_hi), past_hi=past_hi,
                new_lo=rng.randint(0, new_hi), new_hi=new_hi, **options, **heads)


# ---------------------------------------------------------------- inputs

def _lengths(case, seed, lo, hi, salt):
    """Lengths spread evenly from lo to hi, in an order of the seed's (a batch's size is the case's own)."""
    n, a, b = case["requests"], case[lo], case[hi]
    spread = [b if n == 1 else a + (b - a) * i // (n - 1) for i in range(n)]
    order = torch.randperm(n, generator=torch.Generator().manual_seed(seed * 8 + salt)).tolist()
    return [spread[i] for i in order]


def _ceil(a, b):
    return -(-a // b)


def _rope_turns(case):
    """Turns per position of each rotated pair (float64), and the factor on cos and sin."""
    d, theta, f = case["rotary"], 10000.0, case["factor"]
    if case["scaling"] == "base":
        theta = theta * f ** (d / (d - 2))
    t = theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d) / (2 * math.pi)
    if case["scaling"] == "linear":
        t = t / f
    if case["scaling"] == "bands":  # slow pairs are stretched, fast ones kept, a linear blend between
        keep = ((t * 8192 - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        t = t * keep + t / f * (1.0 - keep)
        return t, 0.1 * math.log(f) + 1.0
    return t, 1.0


def _cache(case, lens, g):
    """A pool that holds `lens` tokens' K and V on shuffled pages, and the two block tables."""
    dev, tpp, p = "cuda", case["tpp"], case["page_elems"]
    blocks = [_ceil(n, tpp) for n in lens]
    most = max(max(blocks), 1)
    n_pages = 2 * sum(blocks) + 3
    pool = torch.empty(n_pages * p, dtype=TYPES[case["dtype"]], device=dev)
    step = 1 << 28
    for i in range(0, pool.numel(), step):  # K rows as after a norm, V rows of the same scale
        pool[i:i + step] = torch.randn(min(step, pool.numel() - i), generator=g, device=dev)
    ids = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    row = torch.tensor(blocks, device=dev)
    inside = torch.arange(most, device=dev)[None, :] < row[:, None]
    tables = []
    for part in range(2):
        t = torch.full((len(lens), most), -1, dtype=torch.int32, device=dev)
        t[inside] = ids[part * sum(blocks):(part + 1) * sum(blocks)]
        tables.append(t)
    return pool, n_pages, tables[0], tables[1]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "tables":
        past = _lengths(case, seed, "past_lo", "past_hi", 1)
        new = _lengths(case, seed, "new_lo", "new_hi", 2)
        tpp, planes, rows, width = case["tpp"], case["planes"], case["requests"], case["max_blocks"]
        had = [_ceil(a, tpp) for a in past]
        all_blocks = [_ceil(a + b, tpp) for a, b in zip(past, new)]
        count = [b - a if case["append"] else b for a, b in zip(had, all_blocks)]
        n_new = sum(count) * planes
        n_old = sum(had) * planes if case["append"] else 0
        ids = torch.randperm(n_new + n_old + 5, generator=g, device=dev).to(torch.int32)
        s.update(tokens=sum(new), n_pages=int(ids.numel()), pages=ids[:n_new].contiguous(),
                 past=torch.tensor(past, dtype=torch.int32, device=dev),
                 new=torch.tensor(new, dtype=torch.int32, device=dev), table=None)
        if case["append"]:  # the tables as the steps before left them
            s["table"] = torch.full((planes, rows, width), -1, dtype=torch.int32, device=dev)
            inside = torch.arange(width, device=dev)[None, :] < torch.tensor(had, device=dev)[:, None]
            s["table"][:, inside] = ids[n_new:n_new + n_old].view(planes, -1)
    elif case["op"] == "write":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        kind = TYPES[case["dtype"]]
        packed = torch.randn(t, (hq + 2 * hk) * d, generator=g, device=dev).to(kind)  # one projection's rows
        q, k, v = (x.view(t, -1, d) for x in packed.split([hq * d, hk * d, hk * d], dim=1))
        slots_each = _ceil(t, case["tpp"]) + 2
        n_pages = 2 * slots_each
        order = torch.randperm(n_pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        slots = [order[i * slots_each:][at // case["tpp"]] * case["tpp"] + at % case["tpp"] for i in range(2)]
        turns, factor = _rope_turns(case)
        s.update(q=q, k=k, v=v, q_out=torch.zeros(t, hq, d, dtype=kind, device=dev), n_pages=n_pages,
                 pool=torch.randn(n_pages * case["page_elems"], generator=g, device=dev).to(kind),
                 position=torch.randint(0, case["pos_hi"], (t,), generator=g, device=dev, dtype=torch.int32),
                 k_slots=slots[0], v_slots=slots[1], turns=turns.to(dev), factor=factor,
                 q_weight=None, k_weight=None)
        if case["norm"]:
            s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(kind)
            s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(kind)
    else:
        hq, d, kind = case["q_heads"], case["dim"], TYPES[case["dtype"]]
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
        s["call"] = _bind(s)
    return s


def _bind(s):
    """The library's call on this state, its arguments marshalled once, as a serving loop keeps it."""
    from heterogeneous_lora_amd import runtime
    case = s["case"]
    if case["op"] == "tables":
        cache = runtime.KVCache(None, s["n_pages"], tokens_per_page=case["tpp"])
        s["tables"] = runtime.KVTables(case["planes"], case["requests"], case["max_blocks"], s["tokens"],
                                       table=s["table"])
        return cache.bind_tables(s["tables"], s["pages"], s["past"], s["new"], append=case["append"])
    cache = runtime.KVCache(s["pool"], s["n_pages"], page_elems=case["page_elems"], dtype=case["dtype"],
                            n_kv_heads=case["kv_heads"], head_dim=case["dim"], tokens_per_page=case["tpp"])
    if case["op"] == "write":
        rope = runtime.Rope(case["rotary"], theta=10000.0, interleaved=case["interleaved"],
                            scaling=case["scaling"], factor=case["factor"], original_len=8192,
                            low_turns=1.0, high_turns=4.0, cos_sin_scale=s["factor"])
        return cache.bind_write(s["q"], s["k"], s["v"], s["q_out"], s["position"], s["k_slots"], s["v_slots"],
                                rope=rope, norm=case["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                eps=1e-6)
    options = dict(scale=s["scale"], softcap=case["cap"], window=case["window"], slopes=s["slopes"],
                   prefix_len=s["prefix_len"])
    if case["op"] == "decode":
        return cache.bind_decode(s["q"], s["out"], s["k_table"], s["v_table"], s["seq_len"], **options)
    return cache.bind_prefill(s["q"], s["out"], s["k_table"], s["v_table"], s["seq_len"], s["q_offsets"], **options)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        if op == "tables":
            t = s["tables"]
            return dict(table=t.table, seq_len=t.seq_len, q_offsets=t.q_offsets, token_request=t.token_request,
                        position=t.position, slots=t.slots)
        if op == "write":
            return dict(q=s["q_out"], pool=s["pool"])
        return s["out"]
    if op == "tables":
        return _plain_tables(s)
    if op == "write":
        return _plain_write(s)
    return _plain_attention(s)


def _plain_tables(s):
    case, past, new = s["case"], s["past"].long(), s["new"].long()
    tpp, planes, width = case["tpp"], case["planes"], case["max_blocks"]
    dev = past.device
    seq = past + new
    blocks = (seq + tpp - 1) // tpp
    first = (past + tpp - 1) // tpp if case["append"] else torch.zeros_like(past)
    count = blocks - first
    start = count.cumsum(0) - count
    col = torch.arange(width, device=dev)[None, :]
    here = (col >= first[:, None]) & (col < blocks[:, None])
    ids = s["pages"].view(-1, planes)
    if case["append"]:
        table = s["table"]
        table[:, here] = ids.t()
    elif ids.shape[0] == 0:
        table = torch.full((planes, len(blocks), width), -1, dtype=torch.int32, device=dev)
    else:
        at = (start[:, None] + col).clamp(max=ids.shape[0] - 1)
        table = torch.where(here[:, :, None], ids[at], -1).permute(2, 0, 1).contiguous()
    ends = new.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    tok = torch.arange(s["tokens"], device=dev)
    req = torch.searchsorted(ends, tok, right=True)
    pos = past[req] + tok - offsets[req]
    slots = table[:, req, pos // tpp].long() * tpp + pos % tpp
    return dict(table=table, seq_len=seq.int(), q_offsets=offsets.int(), token_request=req.int(),
                position=pos.int(), slots=slots)


def _plain_write(s):
    case, d, r = s["case"], s["case"]["dim"], s["case"]["rotary"]
    angle = s["position"].double()[:, None] * s["turns"][None, :]
    angle = (angle - angle.floor()) * (2 * math.pi)
    cos = (angle.cos() * s["factor"]).float()[:, None, :]
    sin = (angle.sin() * s["factor"]).float()[:, None, :]

    def turned(x, weight):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        rot, rest = x[..., :r], x[..., r:]
        if case["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([rot, rest], -1)

    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    tpp, width = case["tpp"], case["kv_heads"] * d
    pages = s["pool"].view(s["n_pages"], case["page_elems"])[:, :tpp * width].unflatten(1, (tpp, width))
    for x, slots in ((turned(s["k"], s["k_weight"]), s["k_slots"]), (s["v"], s["v_slots"])):
        pages[slots // tpp, slots % tpp] = x.reshape(-1, width).to(s["pool"].dtype)
    return dict(q=s["q_out"], pool=s["pool"])


def _rows(s, table, r, n):
    """The n cached vectors of request r, [n, kv heads, dim], in 32 bits."""
    case = s["case"]
    tpp, hk, d = case["tpp"], case["kv_heads"], case["dim"]
    pages = s["pool"].view(s["n_pages"], case["page_elems"])
    x = pages[table[r, :_ceil(n, tpp)].long()][:, :tpp * hk * d]
    return x.reshape(-1, hk, d)[:n].float()


def _plain_attention(s):
    case, out = s["case"], s["out"]
    hk, group, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["dim"]
    for r, n in enumerate(s["lens"]):
        a, b = s["offsets"][r], s["offsets"][r + 1]
        if a == b:
            continue
        if n == 0:
            out[a:b] = 0
            continue
        k = _rows(s, s["k_table"], r, n).permute(1, 2, 0).contiguous()
        v = _rows(s, s["v_table"], r, n).transpose(0, 1).contiguous()
        key = torch.arange(n, device=out.device)
        pos = torch.arange(n - (b - a), n, device=out.device)[:, None]
        seen = key <= pos
        if case["window"]:
            seen &= key > pos - case["window"]
        if case["prefix"]:
            seen |= key < case["prefix"]
        few = max(1, int(2e9) // max(1, group * (b - a) * n))  # key heads at once
        for h in range(0, hk, few):
            e = min(h + few, hk)
            q = s["q"][a:b, h * group:e * group].float().view(b - a, e - h, group, d)
            q = q.permute(1, 2, 0, 3).reshape(e - h, group * (b - a), d)
            x = (q @ k[h:e]).view(e - h, group, b - a, n) * s["scale"]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if case["slopes"]:
                x = x + s["slopes"][h * group:e * group].view(e - h, group, 1, 1) * (key - pos)
            x = torch.where(seen, x, -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            x = (x / x.sum(-1, keepdim=True)).view(e - h, group * (b - a), n) @ v[h:e]
            x = x.view(e - h, group, b - a, d).permute(2, 0, 1, 3)
            out[a:b, h * group:e * group] = x.reshape(b - a, -1, d).to(out.dtype)
    return out


# ---------------------------------------------------------------- the work of one pass

def work(case):
    hq, hk, d = case.get("q_heads"), case.get("kv_heads"), case.get("dim")
    if case["op"] == "write":
        t = case["tokens"]
        return dict(bytes=t * (2 * (2 * hq * d + 4 * hk * d) + 20), flops=t * (hq + hk) * (3 * case["rotary"] + 4 * d))
    if case["op"] == "decode":
        lens, new = _lengths(case, 0, "len_lo", "len_hi", 1), [1] * case["requests"]
    else:
        new = _lengths(case, 0, "new_lo", "new_hi", 2)
        lens = [a + b for a, b in zip(_lengths(case, 0, "past_lo", "past_hi", 1), new)]
    if case["op"] == "tables":
        r, p, tpp = case["requests"], case["planes"], case["tpp"]
        ids = p * sum(_ceil(n, tpp) - (_ceil(n - m, tpp) if case["append"] else 0) for n, m in zip(lens, new))
        table = ids if case["append"] else r * p * case["max_blocks"]
        return dict(bytes=4 * (ids + table + 4 * r) + sum(new) * (8 + 8 * p), flops=0)
    w, pre = case["window"], case["prefix"]
    keys = pairs = 0
    for n, m in zip(lens, new):  # keys that some query sees, and seen pairs (a window cuts both)
        keys += min(n, w + m - 1 + pre) if w and m else n if m else 0
        pairs += min(m * (n - m) + m * (m + 1) // 2, m * (w + pre) if w else n * m)
    return dict(bytes=keys * hk * d * 4 + 4 * sum(new) * hq * d, flops=4 * pairs * hq * d)


# ---------------------------------------------------------------- exact results

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_write(s) if case["op"] == "write" else _exact_attention(s)


def _exact_write(s):
    """Each rotated pair as a complex number times e^(2 pi i position turns)."""
    case, r = s["case"], s["case"]["rotary"]
    turns = s["position"].double()[:, None] * s["turns"]
    turns = torch.remainder(turns, 1.0)
    unit = torch.polar(torch.full_like(turns, s["factor"]), 2 * math.pi * turns)[:, None, :]
    result = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + 1e-6) * weight.double()
        y = y.clone()
        if case["interleaved"]:
            first, second = y[..., 0:r:2], y[..., 1:r:2]
        else:
            first, second = y[..., 0:r // 2], y[..., r // 2:r]
        z = torch.complex(first.contiguous(), second.contiguous()) * unit
        first.copy_(z.real)
        second.copy_(z.imag)
        result.append(y)
    pool = s["pool"].double()
    width = case["kv_heads"] * case["dim"]
    for x, slots in ((result[1], s["k_slots"]), (s["v"].double(), s["v_slots"])):
        at = slots // case["tpp"] * case["page_elems"] + slots % case["tpp"] * width
        pool[at[:, None] + torch.arange(width, device=at.device)] = x.reshape(-1, width)
    return dict(q=result[0], pool=pool)


def _exact_attention(s):
    """Head by head and in blocks of queries, in 64 bits."""
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
        inside = (j % tpp)[:, None] * (hk * d) + torch.arange(hk * d, device=out.device)
        base = [t[r].long()[j // tpp] * case["page_elems"] for t in (s["k_table"], s["v_table"])]
        k, v = (s["pool"][at[:, None] + inside].double().view(-1, hk, d) for at in base)
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
