"""Device-memory and stream plumbing around libslora for one workload instance.

PyTorch only allocates device and pinned host memory and provides streams and
events; every step of the LoRA path (allocation bookkeeping, fetch, planning,
shrink, expand) runs in libslora. Used by the tests, the smoke check and the
benchmark.
"""

from __future__ import annotations

from dataclasses import replace as dataclass_replace
from typing import Dict, List, Optional

import numpy as np
import torch

from . import _lib

SENTINEL_I16 = {"f16": 0x7E00, "bf16": 0x7FC0}  # quiet NaN bit patterns (both < 2^15)


def _dev_i16(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device, non_blocking=False)


class HostStore:
    """Adapter weights of one projection set in one pinned host buffer (16-byte aligned rows)."""

    def __init__(self, wl, adapters):
        self.offsets: Dict[tuple, int] = {}
        total = 0
        for a in adapters:
            r = int(wl.ranks[a])
            for p, pr in enumerate(wl.projections):
                for half, L in ((0, pr.d_in), (1, pr.d_out)):
                    self.offsets[(a, p, half)] = total
                    total += ((r * L * 2 + 255) // 256) * 256
        self.buf = torch.empty(max(total, 256), dtype=torch.uint8, pin_memory=True)
        host = self.buf.numpy()
        for a in adapters:
            for p in range(len(wl.projections)):
                at, b = wl.adapter(int(a), p)
                for half, arr in ((0, at), (1, b)):
                    o = self.offsets[(a, p, half)]
                    raw = np.ascontiguousarray(arr).view(np.uint8).ravel()
                    host[o:o + raw.size] = raw
        self.base_ptr = self.buf.data_ptr()

    def ptrs(self, a, n_proj):
        return ([self.base_ptr + self.offsets[(a, p, 0)] for p in range(n_proj)],
                [self.base_ptr + self.offsets[(a, p, 1)] for p in range(n_proj)])


class PagedLoRA:
    """One workload on one GPU: pool, resident adapters, page tables, inputs, workspace."""

    def __init__(self, wl, device: str = "cuda", adapters: Optional[List[int]] = None,
                 fill_kv: bool = True, sentinel: bool = True, pool_seed: Optional[int] = None,
                 store: Optional[HostStore] = None, ordered: bool = False,
                 n_pages: Optional[int] = None):
        """ordered: a pool of its own for the adapters, pages handed out in order (each
        adapter contiguous), no KV pages in it (the split-memory ablation); n_pages then
        defaults to the adapters' pages plus the workload's spare."""
        self.wl = wl
        self.device = torch.device(device)
        P = wl.page_elems
        self.adapters = [int(a) for a in (wl.active_adapters() if adapters is None else adapters)]
        if ordered:
            fill_kv = False
            if n_pages is None:
                n_pages = sum(wl.adapter_pages(a) for a in self.adapters) + 64
        self.n_pages = wl.n_pages if n_pages is None else n_pages
        self.pool_t = torch.empty(self.n_pages * P, dtype=torch.int16, device=self.device)
        if sentinel:
            self.pool_t.fill_(SENTINEL_I16[wl.dtype])
        self.pool = _lib.Pool(self.pool_t.data_ptr(), self.n_pages, P, wl.dtype,
                              wl.pool_seed if pool_seed is None else pool_seed, ordered=ordered)
        d_in = [p.d_in for p in wl.projections]
        d_out = [p.d_out for p in wl.projections]
        for a in self.adapters:
            self.pool.alloc_adapter(a, int(wl.ranks[a]), d_in, d_out)
        self.kv_pages = np.zeros(0, np.int32)
        if fill_kv:
            self._fill_kv()
        self.store = store if store is not None else HostStore(wl, self.adapters)
        self.fetch_ms = self.fetch()
        self.pt_dev, self.pt_len, self.base, self.rank = [], [], [], []
        for p in range(len(wl.projections)):
            pt, base, rank = self.pool.page_table(p, wl.n_adapters)
            self.pt_len.append(int(pt.size))
            self.pt_dev.append(torch.from_numpy(np.ascontiguousarray(pt)).to(self.device)
                               if pt.size else torch.zeros(1, dtype=torch.int32, device=self.device))
            self.base.append(base)
            self.rank.append(rank)
        self.r_max = int(max([int(wl.ranks[a]) for a in self.adapters] + [0]))
        self.r_max = max(self.r_max, 1)

    def _fill_kv(self):
        free = self.pool.info()["n_free"]
        lens = self.wl.kv_seq_lens
        got = []
        if lens.size:
            for L in lens:  # one K and one V page per token, until the pool is full
                n = int(min(2 * int(L), free))
                if n <= 0:
                    break
                got.append(self.pool.alloc_kv(n))
                free -= n
        elif free > 0:
            got.append(self.pool.alloc_kv(free))
        self.kv_pages = np.concatenate(got) if got else np.zeros(0, np.int32)

    def fetch(self, adapters: Optional[List[int]] = None) -> float:
        """Fetch adapters on a side stream; the current stream waits for the done event.
        Returns the fetch time in ms (events on the side stream; waits for it)."""
        side = torch.cuda.Stream(device=self.device)
        done = torch.cuda.Event(enable_timing=True)
        start = torch.cuda.Event(enable_timing=True)
        side.wait_stream(torch.cuda.current_stream(self.device))
        start.record(side)
        done.record(side)  # creates the event so its handle can be passed down
        n_proj = len(self.wl.projections)
        todo = self.adapters if adapters is None else adapters
        rows = [self.store.ptrs(a, n_proj) for a in todo]
        self.pool.fetch_many_async(todo, [r[0] for r in rows], [r[1] for r in rows],
                                   side.cuda_stream, done.cuda_event)
        torch.cuda.current_stream(self.device).wait_event(done)
        self._fetch_done = done
        done.synchronize()
        return start.elapsed_time(done)

    def call(self, proj: int, policy: int = _lib.POLICY_AUTO, wl=None) -> _lib.Call:
        wl = wl or self.wl
        p = wl.projections[proj]
        return _lib.Call(pool_ptr=self.pool_t.data_ptr(), n_pages=self.n_pages,
                         page_elems=wl.page_elems, dtype=wl.dtype, d_in=p.d_in, d_out=p.d_out,
                         page_table_ptr=self.pt_dev[proj].data_ptr(),
                         page_table_len=self.pt_len[proj], base=self.base[proj], rank=wl.ranks,
                         scale=wl.scales.astype(np.float32), r_max=self.r_max,
                         n_tokens=wl.n_tokens, seg_offsets=wl.seg_offsets,
                         seg_adapter=wl.seg_adapter, token_adapter=wl.token_adapter,
                         policy=policy)

    def inputs(self, proj: int):
        """(x, y) device tensors for a projection; y holds y0."""
        return _dev_i16(self.wl.x(proj), self.device), _dev_i16(self.wl.y0(proj), self.device)

    def workspace(self, call: _lib.Call) -> torch.Tensor:
        """Device workspace for calls like `call` (zero-filled once, as the library requires)."""
        return torch.zeros(_lib.workspace_size(call), dtype=torch.uint8, device=self.device)

    def gathered_workspace(self, call: _lib.Call) -> torch.Tensor:
        return torch.zeros(_lib.gathered_workspace_size(call), dtype=torch.uint8, device=self.device)

    def apply_gathered(self, call, x, y, ws, stream=None):
        s = stream or torch.cuda.current_stream(self.device)
        _lib.apply_gathered(call, x.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)

    def apply(self, call: _lib.Call, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
              stream: Optional[torch.cuda.Stream] = None):
        s = stream or torch.cuda.current_stream(self.device)
        _lib.apply(call, x.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)

    def bind_apply(self, call: _lib.Call, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor,
                   stream: Optional[torch.cuda.Stream] = None, gathered: bool = False):
        """apply() (or apply_gathered()) with its arguments marshalled once (a callable
        with no arguments)."""
        s = stream or torch.cuda.current_stream(self.device)
        return _lib.bind_apply(call, x.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
                               s.cuda_stream, gathered=gathered)

    def multi_workspace(self, calls) -> torch.Tensor:
        """Device workspace for apply_multi over `calls` (zero-filled once)."""
        return torch.zeros(_lib.workspace_size_multi(calls), dtype=torch.uint8, device=self.device)

    def bind_apply_multi(self, calls, xs, ys, ws: torch.Tensor,
                         stream: Optional[torch.cuda.Stream] = None):
        """slora_apply_multi over several projections' calls, marshalled once."""
        s = stream or torch.cuda.current_stream(self.device)
        return _lib.bind_apply_multi(calls, [x.data_ptr() for x in xs], [y.data_ptr() for y in ys],
                                     ws.data_ptr(), ws.numel(), s.cuda_stream)

    def shrink(self, call, x, v, ws, stream=None):
        s = stream or torch.cuda.current_stream(self.device)
        _lib.shrink(call, x.data_ptr(), v.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)

    def expand(self, call, v, y, ws, stream=None):
        s = stream or torch.cuda.current_stream(self.device)
        _lib.expand(call, v.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(), s.cuda_stream)

    def close(self):
        torch.cuda.synchronize(self.device)
        self.pool.destroy()


class ServingLoop:
    """Continuous batching of one projection over a unified pool: slora_sched admits
    requests FIFO by free pages, slora_residency keeps adapters resident (LRU eviction),
    adapters a step needs are fetched on a side stream from the host store, and the
    step's batch (new prompts as segments, one decode token per running request) runs
    through slora_apply on the compute stream once the fetch event has fired.

    Everything a step does runs on the stream that is current when the loop is made (or on
    the side stream, ordered with it), whatever stream is current in step().

    Every adapter the workload defines is in the host store; only the pool's pages limit
    how many are resident at once. The weights, x and y0 of a step are seeded synthetic
    data (the same generators the tests and the oracle use)."""

    def __init__(self, wl, n_pages: int, kv_pages_per_token: int = 2, max_batch_tokens: int = 4096,
                 max_running: int = 512, proj: int = 0, device: str = "cuda", seed: int = 0,
                 tokens_per_page: int = 1):
        self.wl, self.proj, self.device = wl, proj, torch.device(device)
        p = wl.projections[proj]
        self.d_in, self.d_out = p.d_in, p.d_out
        self.n_pages = n_pages
        P = wl.page_elems
        self.pool_t = torch.full((n_pages * P,), SENTINEL_I16[wl.dtype], dtype=torch.int16,
                                 device=self.device)
        self.pool = _lib.Pool(self.pool_t.data_ptr(), n_pages, P, wl.dtype, seed)
        self.res = _lib.Residency(self.pool, [p.d_in], [p.d_out])
        self.sched = _lib.Scheduler(self.pool, self.res, kv_pages_per_token, max_batch_tokens,
                                    max_running, tokens_per_page)
        # the projection alone (its weights are drawn as projection 0 of this workload)
        self.one = dataclass_replace(wl, projections=[p], _cache={})
        self.store = HostStore(self.one, list(range(wl.n_adapters)))
        self.side = torch.cuda.Stream(device=self.device)
        self.stream = torch.cuda.current_stream(self.device)
        self.scales = wl.scales.astype(np.float32)
        self.r_max = max(int(wl.ranks.max()), 1)
        self.fetch_bytes = 0
        self.steps_run = 0

    def submit(self, request_id, adapter_id, prompt_len, max_new_tokens, deadline_step=-1):
        r = int(self.wl.ranks[adapter_id]) if adapter_id >= 0 else 0
        self.sched.submit(request_id, adapter_id, r, prompt_len, max_new_tokens, deadline_step)

    def step(self, seed: int):
        """Plan one step, fetch what it needs, run its batch. Returns (batch dict, x, y0, y)
        as host arrays (uint16 bits) for checking, or the batch alone when it is empty."""
        with torch.cuda.stream(self.stream):
            b, x, y0, yd = self._project(seed)
            return b, x, y0, None if yd is None else yd.cpu().numpy().view(np.uint16)

    def _project(self, seed: int):
        """step(), with y left on the device. self.stream is the current stream."""
        b = self.sched.step()
        if b["fetch"].size:
            done = torch.cuda.Event()
            self.side.wait_stream(self.stream)
            ids = [int(a) for a in b["fetch"]]
            rows = [self.store.ptrs(a, 1) for a in ids]
            self.pool.fetch_many_async(ids, [r[0] for r in rows], [r[1] for r in rows],
                                       self.side.cuda_stream, None)
            self.fetch_bytes += sum(int(self.wl.ranks[a]) * (self.d_in + self.d_out) * 2 for a in ids)
            done.record(self.side)
            self.stream.wait_event(done)
        if b["n_tokens"] == 0:
            return b, None, None, None
        pt, base, rank = self.pool.page_table(0, self.wl.n_adapters)
        pt_dev = torch.from_numpy(np.ascontiguousarray(pt)).to(self.device) if pt.size else \
            torch.zeros(1, dtype=torch.int32, device=self.device)
        T = b["n_tokens"]
        rng_x = np.random.default_rng([seed, 1])
        rng_y = np.random.default_rng([seed, 2])
        from workloads import normal_bits
        x = normal_bits(rng_x, (T, self.d_in), 1.0, self.wl.dtype)
        y0 = normal_bits(rng_y, (T, self.d_out), 1.0, self.wl.dtype)
        call = _lib.Call(pool_ptr=self.pool_t.data_ptr(), n_pages=self.n_pages,
                         page_elems=self.wl.page_elems, dtype=self.wl.dtype, d_in=self.d_in,
                         d_out=self.d_out, page_table_ptr=pt_dev.data_ptr(), page_table_len=pt.size,
                         base=base, rank=self.wl.ranks, scale=self.scales, r_max=self.r_max,
                         n_tokens=T, seg_offsets=b["seg_offsets"], seg_adapter=b["seg_adapter"],
                         token_adapter=b["token_adapter"])
        xd = _dev_i16(x, self.device)
        yd = _dev_i16(y0, self.device)
        ws = torch.zeros(_lib.workspace_size(call), dtype=torch.uint8, device=self.device)
        _lib.apply(call, xd.data_ptr(), yd.data_ptr(), ws.data_ptr(), ws.numel(), self.stream.cuda_stream)
        status = _lib.workspace_status(ws.data_ptr(), self.stream.cuda_stream)
        if status:
            raise RuntimeError(f"step {b['step']}: a decode launch gave up waiting")
        self.steps_run += 1
        return b, x, y0, yd

    def close(self):
        torch.cuda.synchronize(self.device)
        self.sched.destroy()
        self.res.destroy()
        self.pool.destroy()


TORCH_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Rope:
    """Rotary positions: frequencies (slora_rope_turns) uploaded once, and the layout.

    scaling: "none", "linear", "base" or "bands" (slora.h); cos_sin_scale multiplies the
    cosines and sines (1 unless the model's scaling asks for another value)."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                 low_turns: float = 1.0, high_turns: float = 4.0, cos_sin_scale: float = 1.0,
                 device: str = "cuda"):
        self.rotary_dim, self.interleaved, self.cos_sin_scale = rotary_dim, interleaved, cos_sin_scale
        self.turns_host = _lib.rope_turns(_lib.Rope(rotary_dim, _lib.ROPE_SCALING[scaling], theta, factor,
                                                    original_len, low_turns, high_turns))
        self.turns = torch.from_numpy(self.turns_host).to(device)


class KVTables:
    """Device arrays slora_kv_tables fills (slora.h, slora_kv_step). table: the tables of the
    steps before, kept and extended by append calls (None: new ones, all -1)."""

    def __init__(self, n_planes: int, n_requests: int, max_blocks: int, n_tokens: int,
                 table: Optional[torch.Tensor] = None, device: str = "cuda"):
        def ints(*shape, dtype=torch.int32):
            return torch.full(shape, -1, dtype=dtype, device=device)
        self.n_planes, self.n_requests, self.max_blocks = n_planes, n_requests, max_blocks
        self.n_tokens = n_tokens
        self.table = ints(n_planes, n_requests, max_blocks) if table is None else table
        _expect("table", self.table, torch.int32, (n_planes, n_requests, max_blocks))
        self.seq_len, self.q_offsets = ints(n_requests), ints(n_requests + 1)
        self.token_request, self.position = ints(n_tokens), ints(n_tokens)
        self.slots = ints(n_planes, n_tokens, dtype=torch.int64)


def _on_gpu(name: str, t: torch.Tensor, device: Optional[torch.device] = None):
    """Kernels follow a tensor's address: one in host memory, or another GPU's, is refused."""
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: expected a tensor on {'the GPU' if device is None else device}, got one on {t.device}")


def _expect(name: str, t: torch.Tensor, dtype, shape, device: Optional[torch.device] = None):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    _on_gpu(name, t, device)


def _opt(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class KVCache:
    """The pool's KV pages as the attention operators see them (slora_kv). bits: of a cached value,
    16 (the cache's type) or 4 (slora.h, "KV cache in 4 bits"; dtype is then that of q, k, v and out).
    In 4 bits the kernels are chosen by what block tables have room for: they need be no wider than the
    longest request (tables of 131072 tokens for requests of 512: twice the time of a decode).

    Each bind_* method checks shapes and types, marshals one call's arguments once and
    returns a no-argument callable; the method of the same name without bind_ makes the call
    at once. Calls go to `stream` (the current stream at binding if None), which the caller
    orders with the work that makes and uses their tensors. A workspace that is not given is
    made, zeroed and, with the bound call, freed on that stream."""

    def __init__(self, pool: Optional[torch.Tensor], n_pages: int, page_elems: int = 0, dtype: str = "f16",
                 n_kv_heads: int = 1, head_dim: int = 8, tokens_per_page: int = 1, bits: int = 16):
        if bits not in (4, 16):
            raise ValueError(f"bits: expected 4 or 16, got {bits}")
        if pool is not None and pool.numel() * pool.element_size() < 2 * n_pages * page_elems:
            raise ValueError(f"pool holds fewer than {n_pages} pages of {page_elems} elements")
        if pool is not None:
            _on_gpu("pool", pool)
            if not pool.is_contiguous():
                raise ValueError("pool: expected a contiguous tensor")
        self.pool, self.n_pages, self.page_elems, self.dtype = pool, n_pages, page_elems, dtype
        self.n_kv_heads, self.head_dim, self.tokens_per_page = n_kv_heads, head_dim, tokens_per_page
        self.device = None if pool is None else pool.device
        self.bits = bits
        four = bits == 4
        self._bind_write = _lib.bind_kv4_write if four else _lib.bind_kv_write
        self._bind_decode = _lib.bind_attn4_decode if four else _lib.bind_attn_decode
        self._bind_prefill = _lib.bind_attn4_prefill if four else _lib.bind_attn_prefill
        self.workspace_size = _lib.attn4_workspace_size if four else _lib.attn_workspace_size

    def _kv(self, n_requests: int = 0, max_blocks: int = 0) -> _lib.KV:
        return _lib.KV(_opt(self.pool), self.n_pages, self.page_elems, _lib.DTYPES[self.dtype],
                       self.n_kv_heads, self.head_dim, self.tokens_per_page, n_requests, max_blocks)

    def _rows(self, name: str, t: torch.Tensor, n: Optional[int] = None, heads: Optional[int] = None):
        """A [rows, heads, head_dim] tensor of the cache's type with a dense last dimension."""
        if t.dtype != TORCH_DTYPES[self.dtype] or t.dim() != 3 or t.shape[2] != self.head_dim or \
                t.stride(2) != 1 or (n is not None and t.shape[0] != n) or \
                (heads is not None and t.shape[1] != heads):
            want = f"[{'rows' if n is None else n}, {'heads' if heads is None else heads}, {self.head_dim}]"
            raise ValueError(f"{name}: expected {TORCH_DTYPES[self.dtype]} {want} with a dense last dimension, "
                             f"got {t.dtype} {tuple(t.shape)}")
        _on_gpu(name, t, self.device)
        return t.data_ptr(), t.stride(0), t.stride(1)

    @staticmethod
    def _stream(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> int:
        return (stream or torch.cuda.current_stream(t.device)).cuda_stream

    # -- block tables, slots, positions (slora_kv_tables)
    def bind_tables(self, tables: KVTables, pages: torch.Tensor, past_len: torch.Tensor,
                    new_len: torch.Tensor, append: bool = False,
                    stream: Optional[torch.cuda.Stream] = None):
        t = tables
        _expect("pages", pages, torch.int32, (pages.numel(),), t.table.device)
        _expect("past_len", past_len, torch.int32, (t.n_requests,), t.table.device)
        _expect("new_len", new_len, torch.int32, (t.n_requests,), t.table.device)
        step = _lib.KVStep(t.n_planes, int(append), pages.data_ptr(), pages.numel(), past_len.data_ptr(),
                           new_len.data_ptr(), t.n_tokens, t.table.data_ptr(), t.seq_len.data_ptr(),
                           t.q_offsets.data_ptr(), t.token_request.data_ptr(), t.position.data_ptr(),
                           t.slots.data_ptr())
        call = _lib.bind_kv_tables(self._kv(t.n_requests, t.max_blocks), step, self._stream(t.table, stream))
        call.tensors = (t, pages, past_len, new_len)
        return call

    def tables(self, *args, **kw):
        self.bind_tables(*args, **kw)()

    # -- norm, rotation, store (slora_kv_write, slora_kv4_write)
    def bind_write(self, q: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                   q_out: torch.Tensor, position: torch.Tensor, k_slots: Optional[torch.Tensor],
                   v_slots: Optional[torch.Tensor], rope: Optional[Rope] = None, norm: bool = False,
                   q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, stream: Optional[torch.cuda.Stream] = None):
        n, hq = q.shape[0], q.shape[1]
        w = _lib.QKV()
        w.n_tokens, w.n_q_heads = n, hq
        w.q, w.q_token_stride, w.q_head_stride = self._rows("q", q)
        w.q_out, w.out_token_stride, w.out_head_stride = self._rows("q_out", q_out, n, hq)
        if k is not None and v is not None:
            w.k, w.k_token_stride, w.k_head_stride = self._rows("k", k, n, self.n_kv_heads)
            w.v, w.v_token_stride, w.v_head_stride = self._rows("v", v, n, self.n_kv_heads)
            for name, s in (("k_slots", k_slots), ("v_slots", v_slots)):
                _expect(name, s, torch.int64, (n,), q.device)
            w.k_slots, w.v_slots = k_slots.data_ptr(), v_slots.data_ptr()
        elif k is not None or v is not None:
            raise ValueError("k and v are given together or not at all")
        _expect("position", position, torch.int32, (n,), q.device)
        w.position = position.data_ptr()
        if rope is not None:
            _expect("rope.turns", rope.turns, torch.float64, (rope.rotary_dim // 2,), q.device)
            w.turns, w.rotary_dim, w.interleaved = rope.turns.data_ptr(), rope.rotary_dim, int(rope.interleaved)
            w.cos_sin_scale = rope.cos_sin_scale
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            if t is not None:
                _expect(name, t, TORCH_DTYPES[self.dtype], (self.head_dim,), q.device)
        w.norm, w.eps, w.q_weight, w.k_weight = int(norm), eps, _opt(q_weight), _opt(k_weight)
        call = self._bind_write(self._kv(), w, self._stream(q, stream))
        call.tensors = (self.pool, q, k, v, q_out, position, k_slots, v_slots, rope, q_weight, k_weight)
        return call

    def write(self, *args, **kw):
        self.bind_write(*args, **kw)()

    # -- K and V of tokens in 16 bits (slora_kv4_read)
    def bind_read(self, k: Optional[torch.Tensor], v: Optional[torch.Tensor], k_slots: Optional[torch.Tensor],
                  v_slots: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream] = None):
        if self.bits != 4:
            raise ValueError("read: the cache's pages hold 16-bit vectors already")
        if (k is None and v is None) or (k is None) != (k_slots is None) or (v is None) != (v_slots is None):
            raise ValueError("read: k with k_slots, v with v_slots, or both")
        r = _lib.KVRows()
        n = (k if k is not None else v).shape[0]
        r.n_tokens = n
        if k is not None:
            r.k, r.k_token_stride, r.k_head_stride = self._rows("k", k, n, self.n_kv_heads)
            _expect("k_slots", k_slots, torch.int64, (n,), k.device)
            r.k_slots = k_slots.data_ptr()
        if v is not None:
            r.v, r.v_token_stride, r.v_head_stride = self._rows("v", v, n, self.n_kv_heads)
            _expect("v_slots", v_slots, torch.int64, (n,), v.device)
            r.v_slots = v_slots.data_ptr()
        call = _lib.bind_kv4_read(self._kv(), r, self._stream(k if k is not None else v, stream))
        call.tensors = (self.pool, k, v, k_slots, v_slots)
        return call

    def read(self, *args, **kw):
        self.bind_read(*args, **kw)()

    # -- attention (slora_attn_decode, slora_attn_prefill and their forms of 4 bits)
    def _attn(self, q, out, k_table, v_table, seq_len, scale, softcap, window, slopes, prefix_len, lse):
        n_req, max_blocks = k_table.shape
        a = _lib.Attn()
        a.n_q_heads = q.shape[1]
        a.scale = self.head_dim ** -0.5 if scale is None else scale
        a.softcap, a.window = softcap, window
        a.q, a.q_token_stride, a.q_head_stride = self._rows("q", q)
        a.out, a.out_token_stride, a.out_head_stride = self._rows("out", out, q.shape[0], q.shape[1])
        _expect("k_table", k_table, torch.int32, (n_req, max_blocks), q.device)
        _expect("v_table", v_table, torch.int32, (n_req, max_blocks), q.device)
        _expect("seq_len", seq_len, torch.int32, (n_req,), q.device)
        if slopes is not None:
            _expect("slopes", slopes, torch.float32, (q.shape[1],), q.device)
        if prefix_len is not None:
            _expect("prefix_len", prefix_len, torch.int32, (n_req,), q.device)
        if lse is not None:
            _expect("lse", lse, torch.float32, (q.shape[0], q.shape[1]), q.device)
        a.k_table, a.v_table, a.seq_len = k_table.data_ptr(), v_table.data_ptr(), seq_len.data_ptr()
        a.slopes, a.prefix_len, a.lse = _opt(slopes), _opt(prefix_len), _opt(lse)
        return a, self._kv(n_req, max_blocks), (self.pool, q, out, k_table, v_table, seq_len, slopes, prefix_len, lse)

    def _ws(self, kv, a, n_tokens, ws, device, stream):
        need = self.workspace_size(kv, a, n_tokens)
        if ws is not None:
            _on_gpu("ws", ws, device)
            if not ws.is_contiguous():
                raise ValueError("ws: expected a contiguous tensor")
            return ws
        with torch.cuda.stream(stream):  # (None: the current one)
            return torch.zeros(need, dtype=torch.uint8, device=device)

    def bind_decode(self, q: torch.Tensor, out: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                    seq_len: torch.Tensor, scale: Optional[float] = None, softcap: float = 0.0,
                    window: int = 0, slopes: Optional[torch.Tensor] = None,
                    prefix_len: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        if q.shape[0] != k_table.shape[0]:
            raise ValueError(f"q: {q.shape[0]} rows for {k_table.shape[0]} requests")
        a, kv, tensors = self._attn(q, out, k_table, v_table, seq_len, scale, softcap, window, slopes,
                                    prefix_len, lse)
        ws = self._ws(kv, a, 0, ws, q.device, stream)
        call = self._bind_decode(kv, a, ws.data_ptr(), ws.nbytes, self._stream(q, stream))
        call.tensors = tensors + (ws,)
        return call

    def decode(self, *args, **kw):
        self.bind_decode(*args, **kw)()

    def bind_prefill(self, q: torch.Tensor, out: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                     seq_len: torch.Tensor, q_offsets: torch.Tensor, scale: Optional[float] = None,
                     softcap: float = 0.0, window: int = 0, slopes: Optional[torch.Tensor] = None,
                     prefix_len: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
        a, kv, tensors = self._attn(q, out, k_table, v_table, seq_len, scale, softcap, window, slopes,
                                    prefix_len, lse)
        _expect("q_offsets", q_offsets, torch.int32, (k_table.shape[0] + 1,), q.device)
        ws = self._ws(kv, a, q.shape[0], ws, q.device, stream)
        call = self._bind_prefill(kv, a, q_offsets.data_ptr(), q.shape[0], ws.data_ptr(), ws.nbytes,
                                  self._stream(q, stream))
        call.tensors = tensors + (q_offsets, ws)
        return call

    def prefill(self, *args, **kw):
        self.bind_prefill(*args, **kw)()


class AttentionLoop(ServingLoop):
    """ServingLoop whose projection makes a layer's packed q, k and v: every step's new
    tokens are normalised, rotated and stored to the KV pages that the scheduler took from
    the unified pool for them, new prompts attend over themselves (slora_attn_prefill) and
    running requests' new tokens over their caches (slora_attn_decode).

    d_out of the projection is (n_q_heads + 2 n_kv_heads) * head_dim; max_len bounds a
    request's cached tokens. attention: softcap, window, slopes, scale as KVCache.bind_decode takes
    them; write: norm, q_weight, k_weight, eps as KVCache.bind_write does. kv_bits: of a cached
    value, 16 or 4; a K page and a V page hold tokens_per_page tokens (None: one in 16 bits, as
    many as fit in 4)."""

    def __init__(self, wl, n_pages: int, n_q_heads: int, n_kv_heads: int, head_dim: int, max_len: int,
                 rope: Optional[Rope] = None, attention: Optional[dict] = None, write: Optional[dict] = None,
                 kv_bits: int = 16, tokens_per_page: Optional[int] = None, **kw):
        if kv_bits not in (4, 16):
            raise ValueError(f"kv_bits: expected 4 or 16, got {kv_bits}")
        token = _lib.kv4_token_bytes(n_kv_heads, head_dim) if kv_bits == 4 else 2 * n_kv_heads * head_dim
        if tokens_per_page is None:
            tokens_per_page = 1 if kv_bits == 16 else max(2 * wl.page_elems // token, 1)
        if tokens_per_page * token > 2 * wl.page_elems:  # (a step would find it, with requests admitted)
            raise ValueError(f"{tokens_per_page} tokens of {token} bytes do not fit a page of {2 * wl.page_elems}")
        super().__init__(wl, n_pages, kv_pages_per_token=2, tokens_per_page=tokens_per_page, **kw)
        if self.d_out != (n_q_heads + 2 * n_kv_heads) * head_dim:
            raise ValueError(f"d_out {self.d_out} is not {n_q_heads} + 2 x {n_kv_heads} heads of {head_dim}")
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.max_len = n_q_heads, n_kv_heads, head_dim, max_len
        self.cache = KVCache(self.pool_t, n_pages, page_elems=wl.page_elems, dtype=wl.dtype,
                             n_kv_heads=n_kv_heads, head_dim=head_dim, tokens_per_page=tokens_per_page,
                             bits=kv_bits)
        self.rope, self.attention, self.write_options = rope, attention or {}, write or {}
        self.cached: Dict[int, int] = {}  # tokens of each running request in the cache
        self.ws: Optional[torch.Tensor] = None

    def _workspace(self, calls, max_blocks: int) -> torch.Tensor:
        """One workspace for every call of the loop, grown as steps need it. calls: (requests,
        prompt tokens) of each, 0 tokens for slora_attn_decode."""
        a = _lib.Attn(n_q_heads=self.n_q_heads)
        need = max(self.cache.workspace_size(self.cache._kv(r, max_blocks), a, n) for r, n in calls)
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        return self.ws

    def submit(self, request_id, adapter_id, prompt_len, max_new_tokens, deadline_step=-1):
        """As ServingLoop.submit. A request's prompt and all but the last of its new tokens are
        cached, at most max_len of them."""
        if prompt_len + max_new_tokens - 1 > self.max_len:
            raise ValueError(f"request {request_id}: a prompt of {prompt_len} and {max_new_tokens} new tokens pass "
                             f"{self.max_len} cached tokens")
        super().submit(request_id, adapter_id, prompt_len, max_new_tokens, deadline_step)

    def step(self, seed: int):
        """One step. Returns (batch dict, qkv, out) with the projections [tokens, heads, head_dim]
        (queries, keys, values) and the attention's output [tokens, n_q_heads, head_dim] on the
        device, in the batch's order: new prompts' tokens, then one of each running request. The
        current stream waits for them."""
        with torch.cuda.stream(self.stream):
            b, qkv, out = self._step(seed)
        user = torch.cuda.current_stream(self.device)
        if out is not None and user != self.stream:
            user.wait_stream(self.stream)
            for t in (qkv, out):
                t.record_stream(user)
        return b, qkv, out

    def _step(self, seed: int):
        b, _, _, y = self._project(seed)
        if y is None:
            self.cached = {}
            return b, None, None
        prompts, running = [int(r) for r in b["seg_request"]], [int(r) for r in b["token_request"]]
        new = np.concatenate([np.diff(b["seg_offsets"]), np.ones(len(running), np.int32)]).astype(np.int32)
        requests = prompts + running
        # a new prompt has nothing cached, also where its id has run before
        past = np.array([0] * len(prompts) + [self.cached[r] for r in running], np.int32)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(self.device)
        pages = np.concatenate([self.sched.request_pages(r) for r in requests])
        T, S, first = b["n_tokens"], len(prompts), int(b["seg_offsets"][-1])
        # tables as wide as the longest request now: kernels and workspaces go by what they have room for
        blocks = -(-int((past + new).max()) // self.cache.tokens_per_page)
        t = KVTables(2, len(requests), blocks, T, device=self.device)
        self.cache.tables(t, dev(pages), dev(past), dev(new))
        hq, hk = self.n_q_heads, self.n_kv_heads
        qkv = y.view(TORCH_DTYPES[self.wl.dtype]).view(T, hq + 2 * hk, self.head_dim)
        q, k, v = qkv.split([hq, hk, hk], dim=1)
        rotated, out = (torch.empty(T, hq, self.head_dim, dtype=qkv.dtype, device=self.device) for _ in range(2))
        self.cache.write(q, k, v, rotated, t.position, t.slots[0], t.slots[1], rope=self.rope, **self.write_options)
        ws = self._workspace([(S, first), (len(running), 0)], blocks)
        if S:
            self.cache.prefill(rotated[:first], out[:first], t.table[0, :S], t.table[1, :S], t.seq_len[:S],
                               t.q_offsets[:S + 1], ws=ws, **self.attention)
        if running:
            self.cache.decode(rotated[first:], out[first:], t.table[0, S:], t.table[1, S:], t.seq_len[S:],
                              ws=ws, **self.attention)
        self.cached = {r: int(n) for r, n in zip(requests, past + new)}  # (a step has every running request)
        return b, qkv, out
