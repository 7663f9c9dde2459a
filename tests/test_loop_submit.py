"""runtime.AttentionLoop.submit refuses a request that its tables could not hold, before the
scheduler knows of it."""

from types import SimpleNamespace

import numpy as np
import pytest

from heterogeneous_lora_amd import runtime as rt


def _loop(max_len):
    loop = rt.AttentionLoop.__new__(rt.AttentionLoop)  # what submit uses of it, without a GPU
    taken = []
    loop.max_len, loop.wl = max_len, SimpleNamespace(ranks=np.array([4, 8]))
    loop.sched = SimpleNamespace(submit=lambda *a: taken.append(a))
    return loop, taken


@pytest.mark.parametrize("prompt,new", [(17, 1), (1, 17), (10, 8), (16, 2)])
def test_refuses_more_than_max_len(prompt, new):
    loop, taken = _loop(16)
    with pytest.raises(ValueError, match="16 cached tokens"):
        loop.submit(5, 1, prompt, new)
    assert taken == []


@pytest.mark.parametrize("prompt,new", [(16, 1), (1, 16), (10, 7)])
def test_takes_what_fits(prompt, new):
    loop, taken = _loop(16)
    loop.submit(5, 1, prompt, new, 9)
    assert taken == [(5, 1, 8, prompt, new, 9)]


@pytest.mark.gpu
def test_the_longest_request_runs_to_its_end():
    from test_gpu_attention_loop import _loop as make
    loop = make(rt, 12 * 3 * 24 + 400)
    loop.submit(0, 3, 70, 11)  # 80 cached tokens, the loop's max_len
    most = 0
    for step in range(12):
        b, _, out = loop.step(seed=step)
        assert out is None or bool(out.isfinite().all())
        most = max([most, *loop.cached.values()])
    assert most == 80 and list(loop.cached) == []
    loop.close()
