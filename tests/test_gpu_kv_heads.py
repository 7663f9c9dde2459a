"""Every head size from 8 to 256 in both attentions and the write: each instance with a last
piece that is full, partly full and empty."""

import numpy as np
import pytest
import torch

import attn_exact as ax
import kv_util as ku
from test_gpu_attention_range import LOST as F16
from test_gpu_attention_weights import LOST as DECODE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", range(8, 257, 8))
def test_attention(d, dtype):
    """Short requests and one whose keys are cut."""
    lens, new = [37, 1700], [37, 5]
    c = ax.dense_cache(lens, dtype=dtype, hk=2, d=d, tpp=2, seed=d)
    g = torch.Generator().manual_seed(d + 1)
    q = torch.randn(sum(new), 4, d, generator=g).to(ku.TORCH[dtype])
    scale = 0.5 * d ** -0.5
    rows = [(r, lens[r] - n + i) for r, n in enumerate(new) for i in range(n)]
    ref = ax.attention(c, q, rows, scale=scale)
    cache, kt, vt = ax.to_gpu(c)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = torch.full((len(rows), 5, d), 7.0, dtype=q.dtype, device="cuda")  # a fifth head that is left alone
    cache.prefill(q.cuda(), out[:, :4], kt, vt, i32(lens), i32([0, 37, 42]), scale=scale)
    ku.check(out[:, :4], ref.out, ax.bound(ref, dtype, *((2.0 ** -8, 0.0) if dtype == "bf16" else F16["prefill"])), "prefill")
    last = [36, 41]
    got = torch.full((2, 5, d), 7.0, dtype=q.dtype, device="cuda")
    cache.decode(q[last].cuda(), got[:, :4], kt, vt, i32(lens), scale=scale)
    lost = DECODE[dtype] if dtype == "bf16" else F16["decode"]
    ku.check(got[:, :4], ref.out[last], ax.bound(ref, dtype, *lost)[last], "decode")
    assert (out[:, 4] == 7).all() and (got[:, 4] == 7).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", range(8, 257, 8))
def test_write(d, interleaved):
    from heterogeneous_lora_amd import runtime as rt
    n, hq, hk = 5, 3, 2
    g = torch.Generator().manual_seed(d)
    q, k, v = (torch.randn(n, h, d, generator=g).bfloat16() for h in (hq, hk, hk))
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g)).bfloat16(), (1 + 0.3 * torch.randn(d, generator=g)).bfloat16()
    pool = torch.randn(2 * n, hk * d, generator=g).bfloat16()
    pos = np.arange(n, dtype=np.int32) * 777
    slots = torch.arange(2 * n).view(2, n)
    for rot in sorted({8, max(d // 2 // 8 * 8, 8), d}):
        rope = rt.Rope(rot, interleaved=interleaved)
        cache = rt.KVCache(pool.cuda(), 2 * n, page_elems=hk * d, dtype="bf16", n_kv_heads=hk, head_dim=d)
        out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
        cache.write(q.cuda(), k.cuda(), v.cuda(), out, torch.from_numpy(pos).cuda(), slots[0].cuda(), slots[1].cuda(),
                    rope=rope, norm=True, q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-5)
        u, tiny = ku.half_step("bf16")
        for x, w, got in ((q, wq, out.cpu()), (k, wk, cache.pool[:n].cpu().view(n, hk, d))):
            y, size = ku.written(x, torch.from_numpy(pos), rope.turns_host, interleaved=interleaved, cos_sin_scale=1.0,
                                 norm=True, eps=1e-5, weight=w)
            ku.check(got, y, u * y.abs() + 2.0 ** -20 * size + tiny, f"rotary {rot}")
        assert torch.equal(cache.pool[n:].cpu().view(n, hk, d), v)
