"""Serving steps over a cache in 4 bits (runtime.AttentionLoop, kv_bits=4): scheduler pages of
several tokens, block tables, write, read and both attentions together, against 64-bit references
that follow each request's tokens."""

import types

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util
import workloads

pytestmark = pytest.mark.gpu
HQ, HK, D = 8, 2, 64


def _loop(n_pages, bits, **kw):
    from heterogeneous_lora_amd import runtime
    wl = workloads.random_small(402, dtype="f16", n_adapters=12, d_in=256, d_out=(HQ + 2 * HK) * D, page_elems=256,
                                n_tokens=1, n_segments=0, rank_choices=(4, 8, 16))
    return runtime.AttentionLoop(wl, n_pages=n_pages, n_q_heads=HQ, n_kv_heads=HK, head_dim=D, max_len=80,
                                 rope=runtime.Rope(D), max_batch_tokens=160, max_running=24, kv_bits=bits, **kw)


def _slots(loop, request, n):
    """K and V slots of a request's n tokens, from its pages (K's and V's of a block together)."""
    tpp = loop.cache.tokens_per_page
    pages = loop.sched.request_pages(request).reshape(-1, 2).astype(np.int64)
    assert len(pages) == -(-n // tpp)
    j = np.arange(n)
    return [torch.from_numpy(pages[j // tpp, i] * tpp + j % tpp).cuda() for i in range(2)]


@pytest.mark.timeout(300)
@pytest.mark.parametrize("bits,tpp,options", [(4, None, dict()), (4, 3, dict(window=9, softcap=20.0)), (16, 2, dict())])
def test_steps_match_references(bits, tpp, options):
    loop = _loop(12 * 3 * 24 + 500, bits, attention=dict(scale=0.2, **options), tokens_per_page=tpp)
    assert loop.cache.tokens_per_page == (tpp or 512 // 80)  # (a token: 2 heads of 2 x 16 + 2 bytes, in 16s)
    rng = np.random.default_rng(5)
    rid = prompts = decoded = 0
    for step in range(14):
        for _ in range(int(rng.poisson(2))):
            loop.submit(rid, int(rng.integers(12)), int(rng.integers(1, 50)), int(rng.integers(2, 12)))
            rid += 1
        had = dict(loop.cached)
        b, qkv, out = loop.step(seed=step)
        if out is None:
            continue
        print(f"step {b['step']}: {b['n_tokens']} tokens", flush=True)
        requests = [int(r) for r in np.concatenate([b["seg_request"], b["token_request"]])]
        S, first = len(b["seg_request"]), int(b["seg_offsets"][-1])
        new = list(np.diff(b["seg_offsets"])) + [1] * b["token_request"].size
        prompts, decoded = prompts + S, decoded + b["token_request"].size
        past = [0 if i < S else had[r] for i, r in enumerate(requests)]
        rows = [(i, past[i] + j) for i, n in enumerate(new) for j in range(int(n))]
        position = torch.tensor([p for _, p in rows], dtype=torch.int32, device="cuda")
        q = torch.empty(len(rows), HQ, D, dtype=torch.float16, device="cuda")
        loop.cache.write(qkv[:, :HQ], None, None, q, position, None, None, rope=loop.rope)
        y, size = util.written(qkv[:, HQ:HQ + HK].cpu(), position.cpu(), loop.rope.turns_host, interleaved=False,
                               cos_sin_scale=1.0, norm=False, eps=0.0, weight=None)
        v = qkv[:, HQ + HK:].cpu()
        kv = []
        for i, r in enumerate(requests):
            n = past[i] + int(new[i])
            at = _slots(loop, r, n)
            if bits == 4:
                held = [torch.empty(n, HK, D, dtype=torch.float16, device="cuda") for _ in range(2)]
                loop.cache.read(*held, *at)
            else:
                pages = loop.pool_t.view(loop.n_pages, -1)[:, :tpp * HK * D].view(torch.float16)
                held = [pages.reshape(-1, HK, D)[s] for s in at]
            kv.append([x.cpu() for x in held])
        k_new, v_new = (torch.stack([kv[i][w][p] for i, p in rows]) for w in range(2))
        if bits == 4:
            assert torch.equal(k_new.double(), four.values(*four.held(y), D))
            assert torch.equal(v_new.double(), four.values(*four.held(v), D))
        else:
            u, tiny = util.half_step("f16")
            util.check(k_new, y, u * y.abs() + 2.0 ** -20 * size + tiny, "stored K")
            assert torch.equal(v_new, v)
        c = types.SimpleNamespace(hk=HK, dtype="f16", lens=[k.shape[0] for k, _ in kv], k=[k for k, _ in kv],
                                  v=[v for _, v in kv])
        ref = dict(scale=0.2, cap=options.get("softcap", 0.0), window=options.get("window", 0))
        if bits == 4:
            want = four.attention(c, q.cpu(), rows, **ref)
            bound = torch.where((torch.arange(len(rows)) < first)[:, None, None], four.bound(want, "f16", False),
                                four.bound(want, "f16", True))
            util.check(out, want.out, bound, f"step {b['step']}")
        else:
            want, bound, _ = util.attention(c, q.cpu(), rows, **ref)
            util.check(out, want, bound, f"step {b['step']}")
    assert prompts >= 10 and decoded >= 30
    assert int(loop.ws[:10240].view(torch.int32).abs().max()) == 0  # counters as they were
    loop.close()


def test_four_bits_hold_more_requests():
    """The same requests in the same small pool: aborted for want of pages in 16 bits, served in 4."""
    aborted, least = [], []
    for bits in (16, 4):
        loop = _loop(900, bits)
        for r in range(12):
            loop.submit(r, r, 13, 20)
        lost, free = 0, []
        for step in range(24):
            b, _, out = loop.step(seed=step)
            lost += b["aborted"].size
            free.append(b["free_pages"])
            assert out is None or bool(torch.isfinite(out).all())
        aborted.append(lost)
        least.append(min(free))
        loop.close()
    assert aborted[0] > 0 and aborted[1] == 0 and least[1] > least[0], (aborted, least)
