"""A cache in 4 bits whose requests share few pages, so that many and long ones are quick to make and to
check: a 64-bit reference of attention of one token (kv4_util's, with its bounds), and how
slora_attn4_decode cuts the keys of a call of many."""

import math
from types import SimpleNamespace

import numpy as np
import torch

import kv4_util as four
from kv_util import TORCH


class Shared:
    """`pages` pages of tokens for K, as many for V, one of each whose tokens are no numbers. Tables draw
    from them; seen(r): the request's keys that its token at the end sees (the others' blocks, where
    none of theirs is seen, are the pages that hold no numbers)."""

    def __init__(self, seed, lens, *, dtype, hk, d, tpp, max_len, pages=24, window=0, prefix=None):
        rng = np.random.default_rng(seed)
        self.dtype, self.hk, self.d, self.tpp, self.lens = dtype, hk, d, tpp, list(lens)
        self.window, self.prefix = window, prefix
        g, sb, size = four.layout(hk, d)
        self.P = -(-tpp * size // 16) * 8
        self.max_blocks = -(-max_len // tpp)
        self.n_pages = 2 * pages + 2
        gen = torch.Generator().manual_seed(seed)
        n = self.n_pages * tpp
        x = torch.randn(n, hk, d, generator=gen, dtype=torch.float64)
        x[-2 * tpp:] = math.nan
        code, step = four.held(x)
        self.x = four.values(code, step, d)  # of place page * tpp + token
        raw = four.token_bytes(code, step, sb)
        self.pool = torch.full((self.n_pages, 2 * self.P), 255, dtype=torch.uint8)
        self.pool[:, :tpp * size] = torch.where(raw < 0, 255, raw).to(torch.uint8).view(self.n_pages, -1)
        shape = (len(lens), self.max_blocks)
        self.kt = rng.integers(0, pages, shape).astype(np.int32)
        self.vt = rng.integers(pages, 2 * pages, shape).astype(np.int32)
        for r, n in enumerate(lens):
            used = np.zeros(self.max_blocks, bool)
            used[np.unique(self.seen(r).numpy() // tpp)] = True
            self.kt[r, ~used], self.vt[r, ~used] = 2 * pages, 2 * pages + 1
            self.kt[r, -(-n // tpp):] = self.vt[r, -(-n // tpp):] = -1

    def seen(self, r):
        n = self.lens[r]
        j = torch.arange(n)
        keep = j >= n - self.window if self.window else j >= 0
        if self.prefix is not None:
            keep = keep | (j < int(self.prefix[r]))
        return j[keep]

    def to_gpu(self):
        from heterogeneous_lora_amd import runtime
        cache = runtime.KVCache(self.pool.cuda(), self.n_pages, page_elems=self.P, dtype=self.dtype, n_kv_heads=self.hk,
                                head_dim=self.d, tokens_per_page=self.tpp, bits=4)
        return cache, torch.from_numpy(self.kt).cuda(), torch.from_numpy(self.vt).cuda()


def attention(c, q, *, scale, cap=0.0, slopes=None):
    """Row r of q sees what request r's last token does: out, mass, total, d, lse as kv4_util's."""
    n, hq, dim = q.shape
    group = hq // c.hk
    out, mass, total = (torch.zeros(n, hq, dim, dtype=torch.float64) for _ in range(3))
    d = torch.zeros(n, hq, 1, dtype=torch.float64)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    clean = torch.nan_to_num(c.x, nan=0.0).transpose(0, 1).contiguous()  # [heads, places, dim]
    places = clean.shape[1]
    far = 2 * c.tpp  # (the places that hold no numbers, at the end)
    for r in range(n):
        j = c.seen(r)
        if not len(j):
            continue
        kp, vp = (torch.from_numpy(t[r].astype(np.int64))[j // c.tpp] * c.tpp + j % c.tpp for t in (c.kt, c.vt))
        assert int(max(kp.max(), vp.max())) < places - far
        x = q[r].double().view(c.hk, group, dim)
        s = torch.bmm(x, clean.transpose(1, 2)).view(hq, places) * scale
        size = torch.bmm(x.abs(), clean.abs().transpose(1, 2)).view(hq, places)[:, kp].amax(1, keepdim=True)
        d[r] = 2.0 ** -24 * (dim + 16) * size * abs(scale)
        s = s[:, kp]
        if cap:
            s = cap * torch.tanh(s / cap)
            d[r] += 2.0 ** -22 * cap if cap <= 256 else 2.0 ** -19 * s.abs().amax(1, keepdim=True)
        if slopes is not None:
            s = s + slopes.double()[:, None] * (j - (c.lens[r] - 1)).double()
        d[r] += 2.0 ** -22 * s.abs().amax(1, keepdim=True)
        lse[r] = torch.logsumexp(s, 1)
        w = torch.exp(s - lse[r][:, None])
        at = torch.zeros(hq, places, dtype=torch.float64).index_add_(1, vp, w).view(c.hk, group, places)
        many = torch.zeros(places, dtype=torch.float64).index_add_(0, vp, torch.ones(len(j), dtype=torch.float64))
        out[r] = torch.bmm(at, clean).view(hq, dim)
        mass[r] = torch.bmm(at, clean.abs()).view(hq, dim)
        total[r] = (many[None, :, None] * clean.abs()).sum(1).repeat_interleave(group, 0)
    return SimpleNamespace(out=out, mass=mass, total=total, d=d, lse=lse)


def cut(c, hq):
    """How the call's keys are cut: KV heads and runs of 32 keys of a wave, units of a workgroup, spans,
    keys of a round, rounds of a span, requests that are cut. spans 0: few keys."""
    hk, group = c.hk, hq // c.hk
    max_len = c.max_blocks * c.tpp
    window = c.window if c.window < max_len else 0
    if len(c.lens) * hk * (window or max_len) < 2500000:
        return SimpleNamespace(spans=0)
    most, room, few = max(16 // group, 1), 7 if c.d > 128 else 16, 3 if c.d > 128 else 5
    heads = min(-(-hk // 4), most, room)
    if heads == 15:
        heads = 16 if most > 15 else 14
    units = -(-hk // heads) * -(-group // 16)
    wg = 4 if units >= 3 else units
    runs = 1 if heads > few or max_len < 1024 else 2 if heads > 1 or c.d > 128 else 4
    spans = -(-(-(-512 // -(-units // wg))) // 8) * 8
    round_ = 128 // wg * runs
    rounds = [max(-(-len(c.seen(r)) // round_), 1) for r in range(len(c.lens))]
    length = -(-sum(rounds) // spans)
    begins = np.concatenate([[0], np.cumsum(rounds)])
    parted = sum(int(a // length != (b - 1) // length) for a, b in zip(begins, begins[1:]))
    return SimpleNamespace(heads=heads, runs=runs, units=wg, spans=spans, round=round_, length=length, cut=parted)
