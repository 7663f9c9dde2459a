"""Plain 64-bit references (CPU) for the KV cache and attention operators, and the bounds
the GPU results are held to.

Bounds. u = finfo(storage type).eps / 2 is one rounding. Attention: the weights are rounded
once (u on each, so at most u * sum_j w_j |v_j| on an output), the output once (u * |out|),
and an error d on a score changes weights by a factor within 1 +- 2d: d is at most
2^-24 (D + 16) max_j scale * sum |q||k_j| for the sum of products (any order) and its
scaling, 2^-22 max_j |s_j| for the roundings in the exponent, and 2^-19 cap for the cap's
exponential and reciprocal. Sums over keys in 32 bits are within 2^-24 * (keys) relative at
worst; 2^-18 covers the lengths tested. Write: one rounding of the result, and 2^-20 of the
rotated pair for the norm's sum (D additions), the angle (2^-25 turns) and the products."""

import math

import numpy as np
import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype):
    f = torch.finfo(TORCH[dtype])
    return f.eps / 2, f.smallest_normal * f.eps / 2


class Cache:
    """A pool on the CPU whose unused places hold NaN, and the block tables of requests."""

    def __init__(self, rng, lens, *, dtype="f16", hk=2, d=64, tpp=1, slack=0, extra=8, blocks_more=1,
                 k_scale=1.0):
        self.dtype, self.hk, self.d, self.tpp, self.lens = dtype, hk, d, tpp, list(lens)
        self.P = tpp * hk * d + slack
        blocks = [-(-n // tpp) for n in lens]
        self.n_pages = 2 * sum(blocks) + extra
        self.max_blocks = max(blocks + [0]) + blocks_more
        g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        self.pool = torch.full((self.n_pages, self.P), float("nan"), dtype=TORCH[dtype])
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.kt = np.full((len(lens), self.max_blocks), -1, np.int32)
        self.vt = self.kt.copy()
        self.k, self.v = [], []
        at = 0
        for r, (n, b) in enumerate(zip(lens, blocks)):
            self.kt[r, :b], self.vt[r, :b] = ids[at:at + b], ids[at + b:at + 2 * b]
            at += 2 * b
            for table, rows, s in ((self.kt, self.k, k_scale), (self.vt, self.v, 1.0)):
                x = (torch.randn(n, hk, d, generator=g) * s).to(TORCH[dtype])
                rows.append(x)
                for j in range(n):
                    o = (j % tpp) * hk * d
                    self.pool[int(table[r, j // tpp]), o:o + hk * d] = x[j].reshape(-1)

    def set_v(self, r, j, value, head=0, dim=0):
        """One element of a cached V vector, in the pool and in the reference's rows."""
        self.v[r][j, head, dim] = value
        self.pool[int(self.vt[r, j // self.tpp]), (j % self.tpp) * self.hk * self.d + head * self.d + dim] = value

    def to_gpu(self):
        from heterogeneous_lora_amd import runtime
        pool = self.pool.cuda()
        cache = runtime.KVCache(pool, self.n_pages, page_elems=self.P, dtype=self.dtype, n_kv_heads=self.hk,
                                head_dim=self.d, tokens_per_page=self.tpp)
        return cache, torch.from_numpy(self.kt).cuda(), torch.from_numpy(self.vt).cuda()


def attention(c, q, rows, *, scale, cap=0.0, window=0, slopes=None, prefix=None):
    """(out, bound, lse) in 64 bits for `rows`: (request, position) of each row of q. Each
    row is computed from the keys it sees alone."""
    n, hq, d = q.shape
    group = hq // c.hk
    u, tiny = half_step(c.dtype)
    out = torch.zeros(n, hq, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    for i, (r, p) in enumerate(rows):
        L = c.lens[r]
        pre = 0 if prefix is None else max(0, int(prefix[r]))
        seen = [j for j in range(L) if (j <= p and (window == 0 or j > p - window)) or j < pre]
        if not seen:
            continue
        kk, vv = c.k[r][seen].double(), c.v[r][seen].double()
        j = torch.tensor(seen, dtype=torch.float64)
        for h in range(hq):
            x = q[i, h].double()
            k, v = kk[:, h // group], vv[:, h // group]
            s = (k @ x) * scale
            err = 2.0 ** -24 * (d + 16) * float((k.abs() @ x.abs()).max()) * abs(scale)
            if cap:
                s = cap * torch.tanh(s / cap)
                err += 2.0 ** -19 * cap
            if slopes is not None:
                s = s + float(slopes[h]) * (j - p)
            err += 2.0 ** -22 * float(s[torch.isfinite(s)].abs().max()) if bool(torch.isfinite(s).any()) else 0.0
            w = torch.softmax(s, 0)
            out[i, h] = w @ v
            bound[i, h] = (u + 2 * err + 2.0 ** -18) * (w @ v.abs()) + u * out[i, h].abs() + tiny
            lse[i, h] = torch.logsumexp(s, 0)
    return out, bound, lse


def check(got, want, bound, what):
    """Elements within their bounds; infinities and NaN where, and only where, expected."""
    got = got.double().cpu()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere than expected"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    off = (got - want).abs()
    excess = torch.where(off == 0, 0.0, off / bound)[finite]  # a row without keys is exact, its bound 0
    worst = float(excess.max()) if excess.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound at {int(excess.argmax())}"
    return worst


def tables(lens_past, lens_new, pages, planes, tpp, max_blocks, n_pages, n_tokens, old=None):
    """slora_kv_tables, token by token. `old`: the tables before, for an append."""
    R = len(lens_past)
    past = [max(int(x), 0) for x in lens_past]
    new = [max(int(x), 0) for x in lens_new]
    table = np.full((planes, R, max_blocks), -1, np.int64) if old is None else old.astype(np.int64).copy()
    req, pos = np.full(n_tokens, -1, np.int64), np.full(n_tokens, -1, np.int64)
    slots = np.full((planes, n_tokens), -1, np.int64)
    at, t = 0, 0
    offsets = []
    for r in range(R):
        offsets.append(min(t, n_tokens))
        first = 0 if old is None else -(-past[r] // tpp)
        for b in range(first, -(-(past[r] + new[r]) // tpp)):
            for p in range(planes):
                if b < max_blocks:
                    table[p, r, b] = pages[at] if at < len(pages) else -1
                at += 1
        for j in range(past[r], past[r] + new[r]):
            if t < n_tokens:
                req[t], pos[t] = r, j
                for p in range(planes):
                    page = table[p, r, j // tpp] if j // tpp < max_blocks else -1
                    if 0 <= page < n_pages:
                        slots[p, t] = page * tpp + j % tpp
            t += 1
    offsets.append(min(t, n_tokens))
    return dict(table=table, seq_len=np.array([a + b for a, b in zip(past, new)], np.int64).reshape(R),
                q_offsets=np.array(offsets), token_request=req, position=pos, slots=slots)


def written(x, position, turns, *, interleaved, cos_sin_scale, norm, eps, weight):
    """q or k as slora_kv_write makes them, in 64 bits, and their bound."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    r = 2 * len(turns)
    a = 2 * math.pi * torch.remainder(position.double()[:, None] * torch.as_tensor(turns)[None, :], 1.0)
    c, s = (torch.cos(a) * cos_sin_scale)[:, None, :], (torch.sin(a) * cos_sin_scale)[:, None, :]
    pair = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    x1, x2 = y[..., pair[0]].clone(), y[..., pair[1]].clone()
    size = y.abs().clone()
    size[..., pair[0]] = size[..., pair[1]] = (x1.abs() + x2.abs()) * abs(cos_sin_scale)
    y = y.clone()
    y[..., pair[0]] = x1 * c - x2 * s
    y[..., pair[1]] = x2 * c + x1 * s
    return y, size
