"""Admission with several tokens to a page (slora_sched_create_paged) against a model of the rules
the header states; host bookkeeping only."""

import ctypes

import numpy as np
import pytest

from heterogeneous_lora_amd import _lib

FAKE_DEV = 0x7F0000000000  # never dereferenced by host code


class Model:
    def __init__(self, free, ppt, tpp, budget, most):
        self.free, self.ppt, self.tpp, self.budget, self.most = free, ppt, tpp, budget, most
        self.queue, self.running = [], []  # [id, prompt, max_new, generated]

    def held(self, q):  # pages of the tokens cached
        return -(-(q[1] + q[3] - 1) // self.tpp) * self.ppt

    def step(self):
        done = [q for q in self.running if q[3] >= q[2]]
        self.running = [q for q in self.running if q[3] < q[2]]
        self.free += sum(map(self.held, done))
        lost = []
        more = lambda q: self.held(q[:3] + [q[3] + 1]) - self.held(q)
        while self.running and self.free < sum(map(more, self.running)):
            q = self.running.pop()
            self.free += self.held(q)
            lost.append(q[0])
        for q in self.running:
            self.free -= more(q)
            q[3] += 1
        decoded = [q[0] for q in self.running]
        tokens, new = len(decoded), []
        while self.queue and len(self.running) < self.most:
            q = self.queue[0]
            if tokens + q[1] > self.budget or self.free < -(-q[1] // self.tpp) * self.ppt:
                break
            self.running.append(self.queue.pop(0))
            q[3] = 1
            self.free -= self.held(q)
            tokens += q[1]
            new.append(q[0])
        return new, decoded, [q[0] for q in done], lost


@pytest.mark.parametrize("tpp", [1, 2, 7, 64])
@pytest.mark.parametrize("ppt", [1, 2, 6])
def test_pages_match_the_rules(ppt, tpp):
    rng = np.random.default_rng(100 * ppt + tpp)
    n_pages = 90 * ppt // tpp + 3 * ppt
    pool = _lib.Pool(FAKE_DEV, n_pages, 64, "f16", 3)
    sched = _lib.Scheduler(pool, None, ppt, 60, 12, tokens_per_page=tpp)
    model = Model(n_pages, ppt, tpp, 60, 12)
    rid = aborts = 0
    for _ in range(200):
        for _ in range(int(rng.poisson(1.0))):
            prompt, new = int(rng.integers(1, 30)), int(rng.integers(1, 25))
            sched.submit(rid, -1, 0, prompt, new)
            model.queue.append([rid, prompt, new, 0])
            rid += 1
        b = sched.step()
        new, decoded, done, lost = model.step()
        assert [int(x) for x in b["seg_request"]] == new
        assert [int(x) for x in b["token_request"]] == decoded
        assert [int(x) for x in b["finished"]] == done
        assert [int(x) for x in b["aborted"]] == lost
        assert b["free_pages"] == model.free
        aborts += len(lost)
        owned = [sched.request_pages(q[0]) for q in model.running]
        assert [p.size for p in owned] == [model.held(q) for q in model.running]
        ids = np.concatenate(owned + [np.empty(0, np.int32)])
        assert np.unique(ids).size == ids.size == n_pages - model.free
    assert aborts > 0 or tpp == 64
    sched.destroy()
    assert pool.n_free() == n_pages
    pool.destroy()


def test_one_token_to_a_page_is_the_plain_scheduler():
    lib = _lib.load()
    traces = []
    for paged in (False, True):
        pool = _lib.Pool(FAKE_DEV, 120, 64, "f16", 3)
        cfg, h = _lib.SchedConfig(2, 60, 12), ctypes.c_void_p()
        tail = (ctypes.c_int32(1), ctypes.byref(h)) if paged else (ctypes.byref(h),)
        make = lib.slora_sched_create_paged if paged else lib.slora_sched_create
        assert make(pool.handle, None, ctypes.byref(cfg), *tail) == _lib.OK
        sched = _lib.Scheduler.__new__(_lib.Scheduler)
        sched._lib, sched.pool, sched.residency, sched.handle = lib, pool, None, h
        rng = np.random.default_rng(9)
        trace = []
        for rid in range(60):
            sched.submit(rid, -1, 0, int(rng.integers(1, 30)), int(rng.integers(1, 25)))
            b = sched.step()
            trace.append([np.asarray(b[k]).tolist() for k in ("seg_request", "token_request", "aborted", "free_pages")]
                         + [sched.request_pages(int(r)).tolist() for r in b["token_request"]])
        traces.append(trace)
        sched.destroy()
        pool.destroy()
    assert traces[0] == traces[1]


@pytest.mark.parametrize("tpp", [0, -1])
def test_refuses_pages_of_no_tokens(tpp):
    with pytest.raises(_lib.SloraError, match="tokens_per_page") as e:
        _lib.Scheduler(_lib.Pool(FAKE_DEV, 8, 64, "f16", 3), None, 2, 8, 4, tokens_per_page=tpp)
    assert e.value.code == _lib.E_INVALID
