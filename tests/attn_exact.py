"""Attention over cached keys in 64 bits (CPU), with what error bounds are made of, for tests
that hold the kernels closer than one rounding of the weights.

A row's result is off by at most
  (weight + 2 d + 2^-18) sum_j w_j |v_j|  +  floor sum_j |v_j|  +  u |out|
weight: the part of a weight that is lost on its way to the product with V; floor: what is
lost whatever the weight, relative to the largest one; d: the error of a score, 2^-24 (D + 16)
max_j scale * sum |q||k_j| for the products, 2^-22 max_j |s_j| for the roundings behind them
and, with a softcap, 2^-22 cap up to 256, 2^-19 max_j |s_j| above; 2^-18: sums over keys in 32 bits; u: half a step of the storage type."""

import math
from types import SimpleNamespace

import numpy as np
import torch

from kv_util import TORCH, half_step


def attention(c, q, rows, *, scale, cap=0.0, window=0, slopes=None, rounded=None):
    """For `rows`, (request, position) of each row of q: out, mass = sum w |v|, total = sum |v|,
    d and lse. rounded: a type that the weights (relative to the largest) are rounded to, as a
    planted mistake."""
    n, hq, dim = q.shape
    group = hq // c.hk
    out, mass, total = (torch.zeros(n, hq, dim, dtype=torch.float64) for _ in range(3))
    d = torch.zeros(n, hq, 1, dtype=torch.float64)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    for i, (r, p) in enumerate(rows):
        j = torch.arange(c.lens[r])
        seen = (j <= p) & ((j > p - window) if window else True)
        if not bool(seen.any()):
            continue
        for h in range(hq):
            k, v, x = c.k[r][seen, h // group].double(), c.v[r][seen, h // group].double(), q[i, h].double()
            s = (k @ x) * scale
            d[i, h] = 2.0 ** -24 * (dim + 16) * float((k.abs() @ x.abs()).max()) * abs(scale)
            if cap:
                s = cap * torch.tanh(s / cap)
                d[i, h] += 2.0 ** -22 * cap if cap <= 256 else 2.0 ** -19 * float(s.abs().max())
            if slopes is not None:
                s = s + float(slopes[h]) * (j[seen].double() - p)
            d[i, h] += 2.0 ** -22 * float(s.abs().max())
            w = torch.exp(s - s.max())
            lse[i, h] = s.max() + torch.log(w.sum())
            z = w.sum()
            if rounded is not None:
                w = w.to(rounded).double()
            out[i, h], mass[i, h], total[i, h] = w @ v / z, w @ v.abs() / z, v.abs().sum(0)
    return SimpleNamespace(out=out, mass=mass, total=total, d=d, lse=lse)


def bound(ref, dtype, weight, floor=0.0):
    u, tiny = half_step(dtype)
    return (weight + 2 * ref.d + 2.0 ** -18) * ref.mass + floor * ref.total + u * ref.out.abs() + tiny


def dense_cache(lens, *, dtype, hk, d, tpp, seed, k=None, v=None):
    """A cache whose requests lie on consecutive pages (long ones are quick to make): what
    kv_util.Cache holds. k, v: the rows of each request, drawn if not given."""
    g = torch.Generator().manual_seed(seed)
    draw = lambda n: torch.randn(n, hk, d, generator=g).to(TORCH[dtype])
    c = SimpleNamespace(dtype=dtype, hk=hk, d=d, tpp=tpp, lens=list(lens), P=tpp * hk * d)
    c.k, c.v = k or [draw(n) for n in lens], v or [draw(n) for n in lens]
    blocks = [-(-n // tpp) for n in lens]
    c.max_blocks, c.n_pages = max(blocks) + 1, 2 * sum(blocks)
    c.kt = np.full((len(lens), c.max_blocks), -1, np.int32)
    c.vt = c.kt.copy()
    c.pool = torch.full((c.n_pages, c.P), float("nan"), dtype=TORCH[dtype])
    at = 0
    for r, b in enumerate(blocks):
        for table, x in ((c.kt, c.k[r]), (c.vt, c.v[r])):
            table[r, :b] = np.arange(at, at + b)
            c.pool[at:at + b].view(-1)[:x.numel()] = x.reshape(-1)
            at += b
    return c


def to_gpu(c):
    from heterogeneous_lora_amd import runtime
    cache = runtime.KVCache(c.pool.cuda(), c.n_pages, page_elems=c.P, dtype=c.dtype, n_kv_heads=c.hk, head_dim=c.d,
                            tokens_per_page=c.tpp)
    return cache, torch.from_numpy(c.kt).cuda(), torch.from_numpy(c.vt).cuda()
