"""Cut attention in a captured graph: counters and partial results over replays with other
lengths, with eager calls in the same workspace between them."""

import pytest
import torch

import attn_exact as ax

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [True, False])
def test_replays_equal_eager_calls(given):
    full = [6000, 900, 3000]
    c = ax.dense_cache(full, dtype="bf16", hk=2, d=128, tpp=4, seed=41)
    cache, kt, vt = ax.to_gpu(c)
    g = torch.Generator().manual_seed(42)
    q = torch.randn(6, 4, 128, generator=g).bfloat16().cuda()
    last = torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seq, offsets = i32(full), i32([0, 1, 4, 6])
    a, b = torch.empty_like(last), torch.empty_like(q)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")

    def bind(a, b, ws):
        return [cache.bind_decode(last, a, kt, vt, seq, ws=ws), cache.bind_prefill(q, b, kt, vt, seq, offsets, ws=ws)]
    last.copy_(q[:3])
    x, y = torch.empty_like(a), torch.empty_like(b)
    eager = bind(x, y, ws)
    for call in eager:
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls = bind(a, b, ws if given else None)
        for call in calls:
            call()
    for turn, lens in enumerate([full, [10, 900, 2999], [5999, 1, 40], [0, 3, 2], full]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(torch.randn(6, 4, 128, generator=g))
        last.copy_(q[:3])
        for call in eager:
            call()
        for t in (a, b):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, x) and torch.equal(b, y), (turn, lens)
    assert int(ws[:10240].view(torch.int32).abs().max()) == 0
