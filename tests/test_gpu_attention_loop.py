"""Serving steps that attend over the unified pool (runtime.AttentionLoop): scheduler pages,
block tables, store and both attentions together, against 64-bit references that follow
each request's tokens."""

import types

import numpy as np
import pytest
import torch

import kv_util as ku
import workloads

pytestmark = pytest.mark.gpu
HQ, HK, D = 8, 2, 64


def _loop(rt, n_pages, **kw):
    wl = workloads.random_small(402, dtype="f16", n_adapters=12, d_in=256, d_out=(HQ + 2 * HK) * D, page_elems=256,
                                n_tokens=1, n_segments=0, rank_choices=(4, 8, 16))
    return rt.AttentionLoop(wl, n_pages=n_pages, n_q_heads=HQ, n_kv_heads=HK, head_dim=D, max_len=80,
                            rope=rt.Rope(D), max_batch_tokens=160, max_running=24, **kw)


def _stored(loop, request, n):
    """K and V of a request's n tokens, from its pages (K and V of a token, token by token)."""
    pages = loop.sched.request_pages(request)
    assert pages.size == 2 * n
    rows = loop.pool_t.view(loop.n_pages, -1)[torch.from_numpy(pages).long().to(loop.device)].cpu()
    rows = rows[:, :HK * D].contiguous().view(torch.float16).view(n, 2, HK, D)
    return rows[:, 0], rows[:, 1]


@pytest.mark.timeout(300)
@pytest.mark.parametrize("options", [dict(), dict(window=9, softcap=20.0)])
def test_steps_match_references(options):
    from heterogeneous_lora_amd import _lib, runtime as rt
    _lib.load()
    loop = _loop(rt, 12 * 3 * 24 + 1200, attention=dict(scale=0.2, **options))
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
        new = list(np.diff(b["seg_offsets"])) + [1] * b["token_request"].size
        prompts, decoded = prompts + len(b["seg_request"]), decoded + b["token_request"].size
        past = [0 if i < len(b["seg_request"]) else had[r] for i, r in enumerate(requests)]
        rows = [(i, past[i] + j) for i, n in enumerate(new) for j in range(int(n))]
        position = torch.tensor([p for _, p in rows], dtype=torch.int32, device="cuda")
        # q as the step rotated it (the same call), V as it came, K within its bound
        q = torch.empty(len(rows), HQ, D, dtype=torch.float16, device="cuda")
        loop.cache.write(qkv[:, :HQ], None, None, q, position, None, None, rope=loop.rope)
        kv = [_stored(loop, r, past[i] + int(new[i])) for i, r in enumerate(requests)]
        y, size = ku.written(qkv[:, HQ:HQ + HK].cpu(), position.cpu(), loop.rope.turns_host, interleaved=False,
                             cos_sin_scale=1.0, norm=False, eps=0.0, weight=None)
        u, tiny = ku.half_step("f16")
        k_new = torch.stack([kv[i][0][p] for i, p in rows])
        v_new = torch.stack([kv[i][1][p] for i, p in rows])
        ku.check(k_new, y, u * y.abs() + 2.0 ** -20 * size + tiny, "stored K")
        assert torch.equal(v_new, qkv[:, HQ + HK:].cpu())
        c = types.SimpleNamespace(hk=HK, dtype="f16", lens=[k.shape[0] for k, _ in kv], k=[k for k, _ in kv],
                                  v=[v for _, v in kv])
        want, bound, _ = ku.attention(c, q.cpu(), rows, scale=0.2, cap=options.get("softcap", 0.0),
                                      window=options.get("window", 0))
        ku.check(out, want, bound, f"step {b['step']}")
    assert prompts >= 10 and decoded >= 30
    assert int(loop.ws[:10240].view(torch.int32).abs().max()) == 0  # counters as they were
    loop.close()


def test_refuses_a_projection_of_another_shape():
    from heterogeneous_lora_amd import runtime as rt
    wl = workloads.random_small(402, dtype="f16", d_in=256, d_out=512, page_elems=256, n_tokens=1, n_segments=0)
    with pytest.raises(ValueError, match="d_out"):
        rt.AttentionLoop(wl, n_pages=64, n_q_heads=8, n_kv_heads=2, head_dim=64, max_len=8)
