"""The write to a cache in 4 bits of so many tokens that a workgroup takes two of them: every byte of
the pool against the 64-bit reference, with tokens that are skipped and slots outside the pool, on the
first and on the second of a pair, and a last workgroup with one."""

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util
from heterogeneous_lora_amd import runtime

N = 4099  # (two to a workgroup from 4096 on)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,hk,hq,d,tpp,rotary,interleaved,norm", [
    ("f16", 2, 4, 64, 3, 64, False, True), ("bf16", 2, 2, 128, 5, 64, True, True), ("bf16", 1, 3, 80, 2, 40, False, False),
    ("f16", 1, 1, 256, 1, 256, True, False), ("bf16", 3, 1, 40, 7, 0, False, True), ("f16", 1, 5, 200, 1, 200, False, True)])
def test_two_tokens_to_a_workgroup(dtype, hk, hq, d, tpp, rotary, interleaved, norm):
    rng = np.random.default_rng(d)
    g, sb, size = four.layout(hk, d)
    P = -(-tpp * size // 16) * 8 + 8
    n_pages = 2 * (-(-N // tpp) + 1)
    gen = torch.Generator().manual_seed(d)
    kind = util.TORCH[dtype]
    packed = torch.randn(N, (hq + 2 * hk) * d, generator=gen).to(kind)
    q, k, v = (x.view(N, -1, d) for x in packed.split([hq * d, hk * d, hk * d], 1))
    order = rng.permutation(n_pages)
    slots = [order[i::2][np.arange(N) // tpp].astype(np.int64) * tpp + np.arange(N) % tpp for i in range(2)]
    position = rng.integers(0, 1 << 20, N).astype(np.int32)
    position[[6, 101, 4096, 4098]] = [-1, -(1 << 31), -5, -1]         # skipped: first, second, both, the last alone
    slots[0][[8, 111, 2000, 2001]] = [-1, n_pages * tpp, 1 << 40, -(1 << 40)]
    slots[1][[9, 110, 2000, 3001]] = [-1, n_pages * tpp + 5, (1 << 63) - 1, 1 << 33]
    slots[0][4097] = -(1 << 63)
    kw = (1 + 0.2 * torch.randn(d, generator=gen)).to(kind) if norm else None
    rope = runtime.Rope(rotary, interleaved=interleaved, cos_sin_scale=1.25) if rotary else None
    pool = torch.from_numpy(rng.integers(0, 256, (n_pages, 2 * P), dtype=np.uint8))
    cache = runtime.KVCache(pool.cuda(), n_pages, page_elems=P, dtype=dtype, n_kv_heads=hk, head_dim=d, tokens_per_page=tpp, bits=4)
    dev = packed.cuda()
    qd, kd, vd = (x.view(N, -1, d) for x in dev.split([hq * d, hk * d, hk * d], 1))
    out = torch.full((N, hq, d), 7.0, dtype=kind, device="cuda")
    weights = dict(q_weight=None if kw is None else kw.cuda(), k_weight=None if kw is None else kw.cuda())
    cache.write(qd, kd, vd, out, torch.from_numpy(position).cuda(), *(torch.from_numpy(s).cuda() for s in slots), rope=rope,
                norm=norm, eps=2.0 ** -20, **weights)
    turns = [] if rope is None else rope.turns_host
    taken = position >= 0
    make = lambda x: util.written(x, torch.from_numpy(position), turns, interleaved=interleaved, cos_sin_scale=1.25, norm=norm,
                                  eps=2.0 ** -20, weight=kw)
    after, expect = cache.pool.cpu().to(torch.int64), pool.to(torch.int64)
    for at, x in ((slots[0], make(k)[0]), (slots[1], v.double())):
        use = taken & (at >= 0) & (at < n_pages * tpp)
        raw = four.token_bytes(*four.held(x[torch.from_numpy(use)]), sb)
        page, cols = torch.from_numpy(at[use] // tpp)[:, None], torch.from_numpy((at[use] % tpp)[:, None] * size + np.arange(size))
        expect[page, cols] = torch.where(raw < 0, after[page, cols], raw)
    assert torch.equal(after, expect), f"{int((after != expect).sum())} bytes differ"
    ref, mass = make(q)
    use = torch.from_numpy(taken)
    u, tiny = util.half_step(dtype)
    util.check(out[use], ref[use], u * ref[use].abs() + 2.0 ** -20 * mass[use] + tiny, "q")
    assert bool((out[~use] == 7.0).all())
