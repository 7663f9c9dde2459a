"""Softcaps of any size: a score's error goes by the score, not by the cap (64-bit references
and bounds of attn_exact)."""

import pytest
import torch

import attn_exact as ax
import kv_util as ku
from test_gpu_attention_range import LOST as F16
from test_gpu_attention_weights import LOST as DECODE

pytestmark = pytest.mark.gpu
LENS, NEW = [150, 33, 1], [20, 33, 1]
CAPS = [1e-30, 0.5, 50.0, 100.0, 256.0, 257.0, 1e3, 1e4, 1e6, 1e12, 1e30, 3e38]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", CAPS)
def test_softcap(cap, slopes, dtype):
    hk, group, d, scale = 2, 2, 64, 1.0
    c = ax.dense_cache(LENS, dtype=dtype, hk=hk, d=d, tpp=3, seed=31)
    g = torch.Generator().manual_seed(32)
    q = torch.randn(sum(NEW), hk * group, d, generator=g).to(ku.TORCH[dtype])
    bias = torch.tensor([0.5, 0.25, 0.125, 0.01]) if slopes else None
    rows = [(r, LENS[r] - n + i) for r, n in enumerate(NEW) for i in range(n)]
    cache, kt, vt = ax.to_gpu(c)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ref = ax.attention(c, q, rows, scale=scale, cap=cap, slopes=bias)
    opts = dict(scale=scale, softcap=cap, slopes=None if bias is None else bias.cuda())
    last = [19, 52, 53]
    for op in ("prefill", "decode"):
        x = q.cuda() if op == "prefill" else q[last].cuda()
        out, lse = torch.empty_like(x), torch.empty(x.shape[:2], device="cuda")
        if op == "prefill":
            cache.prefill(x, out, kt, vt, i32(LENS), i32([0, 20, 53, 54]), lse=lse, **opts)
            lost, want, pick = ((2.0 ** -8, 0.0) if dtype == "bf16" else F16[op]), ref, slice(None)
        else:
            cache.decode(x, out, kt, vt, i32(LENS), lse=lse, **opts)
            lost, want, pick = (DECODE[dtype] if dtype == "bf16" else F16[op]), ref, last
        bound = ax.bound(want, dtype, *lost)[pick]
        worst = ku.check(out, want.out[pick], bound, f"{op}, cap {cap}")
        off = (lse.double().cpu() - want.lse[pick]).abs()
        assert bool((off <= want.d[pick][..., 0] + 2.0 ** -18 + 2.0 ** -22 * want.lse[pick].abs()).all()), (op, float(off.max()))
        print(f"[margin] {op}, cap {cap}: {worst:.3f} of the bound", flush=True)
