"""Attention called on another stream than the current one: its workspace is made and zeroed
in that stream's order, whatever the current stream is busy with."""

import pytest
import torch

import attn_exact as ax

pytestmark = pytest.mark.gpu
HK, GROUP, D = 2, 2, 64
LENS, NEW = [6000, 40, 2500], [3, 2, 1]  # cut keys: counters and partial results are used


@pytest.fixture(scope="module")
def batch():
    c = ax.dense_cache(LENS, dtype="f16", hk=HK, d=D, tpp=4, seed=21)
    cache, kt, vt = ax.to_gpu(c)
    g = torch.Generator().manual_seed(22)
    q = torch.randn(sum(NEW), HK * GROUP, D, generator=g).half().cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seq, offsets = i32(LENS), i32([0, 3, 5, 6])
    last = q[[2, 4, 5]].contiguous()
    def calls(a, b, **kw):
        return (lambda m: getattr(cache, m + "decode")(last, a, kt, vt, seq, **kw),
                lambda m: getattr(cache, m + "prefill")(q, b, kt, vt, seq, offsets, **kw))
    want = torch.empty_like(last), torch.empty_like(q)
    for call in calls(*want):
        call("")
    torch.cuda.synchronize()
    return calls, want


def busy():
    """Some tens of milliseconds of work on the current stream."""
    x = torch.randn(4096, 4096, device="cuda")
    for _ in range(40):
        x = x @ x
        x = x / x.norm()
    return x


def stain(stream):
    """Memory as an earlier user may have left it, back in the stream's pool."""
    with torch.cuda.stream(stream):
        for size in (1 << 20, 8 << 20, 64 << 20):
            torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("bound", [False, True])
def test_workspace_is_ordered_with_its_stream(batch, bound):
    calls, want = batch
    side = torch.cuda.Stream()
    for turn in range(3):
        got = [torch.full_like(x, 7.0) for x in want]
        stain(side)
        stain(torch.cuda.current_stream())
        side.wait_stream(torch.cuda.current_stream())
        keep = busy()
        for call in calls(*got, stream=side):
            if bound:
                run = call("bind_")
                run()
                del run  # its workspace goes back while the kernel may still run
            else:
                call("")
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), turn
        torch.cuda.synchronize()
        del keep


def test_freed_workspace_is_not_reused_early(batch):
    """A workspace freed with its bound call goes back to the stream that reads it: work queued
    there afterwards may take it, work of the current stream may not."""
    calls, want = batch
    side = torch.cuda.Stream()
    got = [torch.full_like(x, 7.0) for x in want]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = busy()  # the calls wait for this
    for call in calls(*got, stream=side):
        call("")
    stain(torch.cuda.current_stream())
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    del keep
