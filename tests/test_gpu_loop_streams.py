"""Serving loops stepped under another stream than their own: every launch goes to the loop's
stream, and the caller's stream waits for what it is given."""

import numpy as np
import pytest
import torch

import workloads
from test_gpu_attention_loop import D, HK, HQ, _loop
from test_gpu_kv_streams import busy

pytestmark = pytest.mark.gpu


@pytest.fixture
def launches(monkeypatch):
    """Streams of the loop's launches, by entry point."""
    from heterogeneous_lora_amd import _lib
    seen = []

    def watch(name, at):
        real = getattr(_lib, name)

        def call(*args):
            seen.append((name, int(args[at])))
            return real(*args)
        monkeypatch.setattr(_lib, name, call)
    for name in ("apply", "bind_kv_tables", "bind_kv_write", "bind_attn_decode", "bind_attn_prefill"):
        watch(name, -1)
    return seen


def _submit(loop):
    rng = np.random.default_rng(3)
    for r in range(12):
        loop.submit(r, int(rng.integers(12)), int(rng.integers(1, 40)), int(rng.integers(2, 9)))


def test_attention_loop_under_another_stream(launches):
    from heterogeneous_lora_amd import runtime as rt
    own = torch.cuda.Stream()
    with torch.cuda.stream(own):
        loop = _loop(rt, 12 * 3 * 24 + 400, attention=dict(scale=0.2))
    plain = _loop(rt, 12 * 3 * 24 + 400, attention=dict(scale=0.2))
    _submit(loop)
    _submit(plain)
    wanted = []
    for step in range(6):
        _, _, out = plain.step(seed=step)
        wanted.append(None if out is None else out.clone())
    torch.cuda.synchronize()
    assert {s for _, s in launches} == {torch.cuda.current_stream().cuda_stream}
    del launches[:]
    user = torch.cuda.Stream()
    with torch.cuda.stream(user):
        for step in range(6):
            keep = busy()
            _, qkv, out = loop.step(seed=step)
            copy = None if out is None else out * 1  # on the user's stream, which waits for the step
            user.synchronize()
            assert (copy is None) == (wanted[step] is None)
            assert copy is None or torch.equal(copy, wanted[step])
            del keep
    assert {n for n, _ in launches} == {"apply", "bind_kv_tables", "bind_kv_write", "bind_attn_decode", "bind_attn_prefill"}
    assert {s for _, s in launches} == {own.cuda_stream}
    loop.close()
    plain.close()


def test_serving_loop_under_another_stream(launches):
    from heterogeneous_lora_amd import runtime as rt
    wl = workloads.random_small(402, dtype="f16", n_adapters=12, d_in=256, d_out=(HQ + 2 * HK) * D, page_elems=256,
                                n_tokens=1, n_segments=0, rank_choices=(4, 8, 16))
    results = []
    for user in (torch.cuda.current_stream(), torch.cuda.Stream()):
        loop = rt.ServingLoop(wl, n_pages=12 * 3 * 24 + 400, max_batch_tokens=160, max_running=24)
        own = torch.cuda.current_stream().cuda_stream
        _submit(loop)
        with torch.cuda.stream(user):
            results.append([loop.step(seed=i)[3] for i in range(4)])
        assert {s for _, s in launches} == {own}
        del launches[:]
        loop.close()
    for a, b in zip(*results):
        assert (a is None) == (b is None) and (a is None or np.array_equal(a, b))
