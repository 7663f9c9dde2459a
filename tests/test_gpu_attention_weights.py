"""Attention's weights on their way to the product with V: decode keeps them past the storage
type's bits (64-bit references and bounds of attn_exact)."""

import pytest
import torch

import attn_exact as ax
import kv_util as ku

DECODE = {  # scores are small, so that the bound is made of the weights' and the result's rounding
    "one chunk": dict(lens=[40, 33, 7], hk=2, group=2, d=64),
    "heads of 128": dict(lens=[50], hk=4, group=1, d=128),
    "heads of 256": dict(lens=[60, 90], hk=1, group=4, d=256),
    "cut": dict(lens=[1500, 700], hk=1, group=2, d=96),
    "heads to waves": dict(lens=[30 + i % 9 for i in range(260)], hk=4, group=1, d=64),
}
# of a weight, and of the largest: bf16 has 2^-8 and 2^-7 of the cut-off rest; f16 2^-11 and
# 2^-10 and its smallest value
LOST = {"bf16": (2.0 ** -15, 0.0), "f16": (2.0 ** -21, 2.0 ** -24)}


def decode_case(name, dtype):
    spec = DECODE[name]
    c = ax.dense_cache(spec["lens"], dtype=dtype, hk=spec["hk"], d=spec["d"], tpp=2, seed=11)
    q = torch.randn(len(c.lens), c.hk * spec["group"], c.d, generator=torch.Generator().manual_seed(12))
    return c, q.to(ku.TORCH[dtype]), [(r, n - 1) for r, n in enumerate(c.lens)], 0.01


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode(name, dtype):
    c, q, rows, scale = decode_case(name, dtype)
    cache, kt, vt = ax.to_gpu(c)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    cache.decode(q.cuda(), out, kt, vt, torch.tensor(c.lens, dtype=torch.int32, device="cuda"), scale=scale)
    ref = ax.attention(c, q, rows, scale=scale)
    worst = ku.check(out, ref.out, ax.bound(ref, dtype, *LOST[dtype]), f"{name} {dtype}")
    print(f"[margin] {name} {dtype}: {worst:.3f} of the bound", flush=True)
