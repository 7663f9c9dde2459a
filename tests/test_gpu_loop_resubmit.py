"""A request id that the client ended (slora_sched_finish) may be submitted again: its new
prompt starts with nothing cached."""

import pytest
import torch

from test_gpu_attention_loop import _loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("between", [0, 1])
def test_id_of_an_ended_request(between):
    from heterogeneous_lora_amd import runtime as rt
    pages = 12 * 3 * 24 + 400
    loop, fresh = _loop(rt, pages), _loop(rt, pages)
    loop.submit(7, 2, 30, 9)
    loop.step(seed=0)
    loop.step(seed=1)
    loop.sched.finish(7)
    for _ in range(between):  # a step in which nothing runs
        assert loop.step(seed=2)[2] is None
    for x in (loop, fresh):
        x.submit(7, 4, 12, 5)
    for seed in (5, 6, 7):
        _, _, got = loop.step(seed=seed)
        _, _, want = fresh.step(seed=seed)
        assert torch.equal(got, want)
        assert loop.cached == fresh.cached == {7: 12 + seed - 5}
    loop.close()
    fresh.close()
