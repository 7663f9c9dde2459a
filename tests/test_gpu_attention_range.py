"""f16 weights over long caches: a tail of keys, each far below a key that dominates, weighs as
much as it should (64-bit references and bounds of attn_exact)."""

import pytest
import torch

import attn_exact as ax
import kv_util as ku

D, SCALE = 64, 0.01
# of a weight, and of the largest: decode's two values, prefill's one; subnormals from 2^-14 on,
# with the largest weight at 2^7 or above
LOST = {"decode": (2.0 ** -21, 2.0 ** -31), "prefill": (2.0 ** -11, 2.0 ** -32)}


def case(n, top, dtype="f16", spread=1.5):
    """One request of n keys, two query heads on one: its scores are `top[j]` at key j and within
    -spread .. spread elsewhere (nats). V is 0 at the keys of `top`, around 1 elsewhere."""
    g = torch.Generator().manual_seed(n)
    x = torch.randn(D, generator=g)
    x *= 10 / x.norm()                      # x.x * SCALE = 1
    t = (torch.rand(n, generator=g) * 2 - 1) * spread
    for j, s in top.items():
        t[j] = s
    k = (t[:, None] * x + 0.1 * torch.randn(n, D, generator=g)).to(ku.TORCH[dtype]).view(n, 1, D)
    v = 1 + 0.5 * torch.randn(n, 1, D, generator=g)
    v[list(top)] = 0
    c = ax.dense_cache([n], dtype=dtype, hk=1, d=D, tpp=16, seed=0, k=[k], v=[v.to(ku.TORCH[dtype])])
    q = (x + 0.01 * torch.randn(1, 2, D, generator=g)).to(ku.TORCH[dtype])
    return c, q


CASES = {
    "first key dominates": (131072, {0: 18.5}),
    "last key dominates": (131072, {131071: 18.5}),
    "short": (3000, {5: 16.0}),
    # the maximum moves when it has grown by 8 log 2: just below it the weights are largest
    "maximum lags": (900, {100: 5.4 + 1.5, 500: 5.4 + 1.5}),
    "maximum moves": (900, {100: 5.8 + 1.5, 500: 14.0}),
}


@pytest.mark.parametrize("name", ["first key dominates", "last key dominates", "short"])
def test_bound_notices_unscaled_weights(name):
    """On the CPU: weights rounded to f16 with the largest at 1 lose the tail."""
    c, q = case(*CASES[name])
    rows = [(0, c.lens[0] - 1)]
    ref = ax.attention(c, q, rows, scale=SCALE)
    flat = ax.attention(c, q, rows, scale=SCALE, rounded=torch.float16)
    for lost in LOST.values():
        with pytest.raises(AssertionError, match="times the bound"):
            ku.check(flat.out, ref.out, ax.bound(ref, "f16", *lost), name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_tail_keeps_its_weight(name):
    c, q = case(*CASES[name])
    n = c.lens[0]
    cache, kt, vt = ax.to_gpu(c)
    seq = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, 2, device="cuda")
    rows = [(0, n - 1)]
    ref = ax.attention(c, q, rows, scale=SCALE)
    for op in ("decode", "prefill"):
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        if op == "decode":
            cache.decode(q.cuda(), out, kt, vt, seq, scale=SCALE, lse=lse)
        else:
            offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
            cache.prefill(q.cuda(), out, kt, vt, seq, offsets, scale=SCALE, lse=lse)
        worst = ku.check(out, ref.out, ax.bound(ref, "f16", *LOST[op]), f"{op} {name}")
        assert float((lse.double().cpu() - ref.lse).abs().max()) < 1e-4, op
        print(f"[margin] {op} {name}: {worst:.3f} of the bound", flush=True)


@pytest.mark.gpu
def test_prompt_rows_keep_their_tails():
    """Rows of whole tiles (not cut), a dominating key in front of each row's tail."""
    n, new = 6000, 600
    c, q1 = case(n, {0: 17.0})
    g = torch.Generator().manual_seed(1)
    q = (q1 + 0.01 * torch.randn(new, 2, D, generator=g)).to(torch.float16)
    cache, kt, vt = ax.to_gpu(c)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.prefill(q.cuda(), out, kt, vt, i32(n), i32(0, new), scale=SCALE)
    some = list(range(0, new, 37)) + [new - 1]
    ref = ax.attention(c, q[some], [(0, n - new + i) for i in some], scale=SCALE)
    ku.check(out.cpu()[some], ref.out, ax.bound(ref, "f16", *LOST["prefill"]), "prompt")
