"""Plain 64-bit references (CPU) for the cache in 4 bits: what a group of 32 dimensions is held
as, a token's bytes, attention over the values held, and the bounds the GPU results are held to.

The values held are exact in both storage types, so attention's bounds are those of its own
arithmetic. u = finfo(storage type).eps / 2 is one rounding of the result. A row is off by at most
  (weight + 2 d + 2^-18) sum_j w_j |v_j|  +  floor sum_j |v_j|  +  u |out|
weight, floor: what a weight loses on its way to the product with V, which takes f16 whatever the
storage type: 2^-11 of it and 2^-32 of the largest where it is rounded once, 2^-21 and 2^-31 where
it goes in as two values (slora_attn4_decode with f16 q); long prompts with bf16 q round it to bf16. d: the error of a score: 2^-24 (D + 16)
max_j scale sum |q||k_j| for the products in any order and their scaling, 2^-22 max_j |s_j| for
the roundings behind them, with a softcap 2^-22 of it up to 256 and 2^-19 max_j |s_j| above.
2^-18: sums over keys in 32 bits."""

import math
from types import SimpleNamespace

import numpy as np
import torch

from kv_util import TORCH, half_step

LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
NAN_STEP, MAX_STEP = 255, 226
STEPS = torch.from_numpy((np.arange(MAX_STEP + 1, dtype=np.uint16) << 7).view(np.float16).astype(np.float64))


def layout(hk, d):
    """Groups of a head, bytes of its steps, bytes of a token."""
    g = -(-d // 32)
    sb = next(x for x in (1, 2, 4, 8) if x >= g)
    return g, sb, -(-hk * (16 * g + sb) // 16) * 16


def nearest(x, marks):
    """Index of the mark nearest to x (>= 0), of two equally near the even one."""
    mids = (marks[1:] + marks[:-1]) / 2
    n = torch.searchsorted(mids, x.contiguous())
    tie = (n < len(mids)) & (mids[n.clamp(max=len(mids) - 1)] == x)
    return torch.where(tie & (n % 2 == 1), n + 1, n)


def held(x):
    """Codes [..., G, 32] and step bytes [..., G] of [..., d] values."""
    d = x.shape[-1]
    g = -(-d // 32)
    x = torch.nn.functional.pad(x.double(), (0, 32 * g - d)).unflatten(-1, (g, 32))
    most = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    most = torch.where(bad, 0.0, most)
    step = nearest(most, 6 * STEPS)
    size = STEPS[step][..., None]
    t = torch.where(size == 0, 0.0, torch.nan_to_num(x.abs()) / torch.where(size == 0, 1.0, size))
    code = nearest(t, LEVELS) + torch.where(torch.signbit(x), 8, 0)
    return torch.where(bad[..., None], 0, code), torch.where(bad, NAN_STEP, step)


def values(code, step, d):
    """The values codes and steps stand for, [..., d], 64 bits."""
    size = torch.where(step == NAN_STEP, math.nan, STEPS[step.clamp(max=MAX_STEP)])
    v = LEVELS[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    return (v * size[..., None]).flatten(-2)[..., :d]


def token_bytes(code, step, sb):
    """[n, hk, G, 32] codes and [n, hk, G] steps as tokens' bytes [n, bytes]; -1: not written."""
    n, hk, g, _ = code.shape
    size = layout(hk, 32 * g)[2]
    out = torch.full((n, size), -1, dtype=torch.int64)
    pair = code.view(n, hk, g, 4, 4, 2)
    byte = (pair[..., 0] | pair[..., 1] << 4).transpose(2, 3)  # [n, hk, 4, g, 4]
    out[:, :hk * 16 * g] = byte.reshape(n, -1)
    steps = torch.zeros(n, hk, sb, dtype=torch.int64)
    steps[:, :, :g] = step
    out[:, hk * 16 * g:hk * (16 * g + sb)] = steps.view(n, -1)
    return out


class Cache:
    """A pool on the CPU whose unused bytes are 255 (steps that are no numbers), the block tables of
    requests, and k, v: the values its tokens hold, exact in the storage type."""

    def __init__(self, rng, lens, *, dtype="f16", hk=2, d=64, tpp=1, slack=0, extra=8, blocks_more=1, k_scale=1.0,
                 v_scale=1.0, shuffle=True):
        self.dtype, self.hk, self.d, self.tpp, self.lens = dtype, hk, d, tpp, list(lens)
        self.g, self.sb, self.size = layout(hk, d)
        self.P = -(-tpp * self.size // 16) * 8 + slack
        blocks = [-(-n // tpp) for n in lens]
        self.n_pages = 2 * sum(blocks) + extra
        self.max_blocks = max(blocks + [0]) + blocks_more
        gen = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        self.pool = torch.full((self.n_pages, 2 * self.P), 255, dtype=torch.uint8)
        ids = (rng.permutation(self.n_pages) if shuffle else np.arange(self.n_pages)).astype(np.int32)
        self.kt = np.full((len(lens), self.max_blocks), -1, np.int32)
        self.vt = self.kt.copy()
        self.k, self.v = [], []
        at = 0
        for r, (n, b) in enumerate(zip(lens, blocks)):
            self.kt[r, :b], self.vt[r, :b] = ids[at:at + b], ids[at + b:at + 2 * b]
            at += 2 * b
            for which, rows, s in ((0, self.k, k_scale), (1, self.v, v_scale)):
                rows.append(torch.zeros(n, hk, d, dtype=TORCH[dtype]))
                if n:
                    self.put(r, slice(0, n), which, torch.randn(n, hk, d, generator=gen, dtype=torch.float64) * s)

    def put(self, r, tokens, which, x):
        """Stores x [n, hk, d] as the K (which 0) or V (1) of `tokens` of request r."""
        code, step = held(x)
        v = values(code, step, self.d)
        rows = (self.k, self.v)[which][r]
        rows[tokens] = v.to(rows.dtype)
        assert torch.equal(torch.nan_to_num(rows[tokens].double(), nan=-7.0), torch.nan_to_num(v, nan=-7.0))
        raw = token_bytes(code, step, self.sb)
        raw = torch.where(raw < 0, 255, raw).to(torch.uint8)
        j = torch.arange(self.lens[r])[tokens].numpy()
        table = (self.kt, self.vt)[which][r]
        at = torch.from_numpy((j % self.tpp)[:, None] * self.size + np.arange(self.size))
        self.pool[torch.from_numpy(table[j // self.tpp].astype(np.int64))[:, None], at] = raw

    def to_gpu(self):
        from heterogeneous_lora_amd import runtime
        cache = runtime.KVCache(self.pool.cuda(), self.n_pages, page_elems=self.P, dtype=self.dtype,
                                n_kv_heads=self.hk, head_dim=self.d, tokens_per_page=self.tpp, bits=4)
        return cache, torch.from_numpy(self.kt).cuda(), torch.from_numpy(self.vt).cuda()


def attention(c, q, rows, *, scale, cap=0.0, window=0, slopes=None, prefix=None, rounded=None):
    """For `rows`, (request, position) of each row of q: out, mass = sum w |v|, total = sum |v|,
    d and lse, each row from the keys it sees alone. rounded: a type that the weights (relative to the
    largest) are rounded to, as a planted mistake."""
    n, hq, dim = q.shape
    group = hq // c.hk
    out, mass, total = (torch.zeros(n, hq, dim, dtype=torch.float64) for _ in range(3))
    d = torch.zeros(n, hq, 1, dtype=torch.float64)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64)
    wide = {r: (c.k[r].double().transpose(0, 1), c.v[r].double().transpose(0, 1)) for r in {r for r, _ in rows}}
    for i, (r, p) in enumerate(rows):
        j = torch.arange(c.lens[r])
        seen = (j <= p) & ((j > p - window) if window else True)
        if prefix is not None:
            seen |= j < int(prefix[r])
        if not bool(seen.any()):
            continue
        k, v = (x[:, seen].repeat_interleave(group, 0) for x in wide[r])  # [hq, keys, dim]
        x = q[i].double()
        s = (k @ x[:, :, None])[..., 0] * scale
        d[i] = 2.0 ** -24 * (dim + 16) * (k.abs() @ x.abs()[:, :, None])[..., 0].amax(-1, keepdim=True) * abs(scale)
        if cap:
            s = cap * torch.tanh(s / cap)
            d[i] += 2.0 ** -22 * cap if cap <= 256 else 2.0 ** -19 * s.abs().amax(-1, keepdim=True)
        if slopes is not None:
            s = s + slopes.double()[:, None] * (j[seen].double() - p)
        d[i] += 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
        w = torch.exp(s - s.amax(-1, keepdim=True))
        z = w.sum(-1, keepdim=True)
        lse[i] = torch.logsumexp(s, -1)
        if rounded is not None:
            w = w.to(rounded).double()
        w = (w / z)[:, None]
        out[i], mass[i], total[i] = (w @ v)[:, 0], (w @ v.abs())[:, 0], v.abs().sum(1)
    return SimpleNamespace(out=out, mass=mass, total=total, d=d, lse=lse)


def bound(ref, dtype, decode, back=False):
    """back: keys were read back to the storage type first (long prompts), weights are then of it."""
    u, tiny = half_step(dtype)
    weight, floor = (2.0 ** -21, 2.0 ** -31) if decode and dtype == "f16" else (2.0 ** -11, 2.0 ** -32)
    if back and dtype == "bf16":
        weight, floor = u, 0.0
    return (weight + 2 * ref.d + 2.0 ** -18) * ref.mass + floor * ref.total + u * ref.out.abs() + tiny
