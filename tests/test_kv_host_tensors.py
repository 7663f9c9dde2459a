"""Tensors in host memory are refused before any call (a kernel would follow their address)."""

import pytest
import torch

from heterogeneous_lora_amd import _lib, runtime as rt


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _lib.load()


def _cache():
    return rt.KVCache(None, 8, page_elems=128, n_kv_heads=2, head_dim=64)


def test_host_tables_and_pool():
    with pytest.raises(ValueError, match="table: expected a tensor on the GPU"):
        rt.KVTables(2, 3, 4, 5, device="cpu")
    with pytest.raises(ValueError, match="pool: expected a tensor on the GPU"):
        rt.KVCache(torch.zeros(1024, dtype=torch.float16), 8, page_elems=128, n_kv_heads=2, head_dim=64)


def test_host_rows():
    q = torch.zeros(1, 4, 64, dtype=torch.float16)
    table, i32 = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bind in (lambda: _cache().bind_decode(q, q, table, table, i32[:1]),
                 lambda: _cache().bind_prefill(q, q, table, table, i32[:1], i32),
                 lambda: _cache().bind_write(q, None, None, q, i32[:1], None, None)):
        with pytest.raises(ValueError, match="q: expected a tensor on the GPU"):
            bind()


@pytest.mark.gpu
def test_every_host_tensor_is_refused():
    """Each tensor of each call in turn, the others where they should be."""
    dev = "cuda"
    pool = torch.zeros(8 * 128, dtype=torch.float16, device=dev)
    cache = rt.KVCache(pool, 8, page_elems=128, n_kv_heads=2, head_dim=64)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)
    half = lambda *s: torch.zeros(*s, dtype=torch.float16, device=dev)
    t = rt.KVTables(2, 1, 4, 1)
    attn = dict(q=half(1, 4, 64), out=half(1, 4, 64), k_table=i32(1, 4), v_table=i32(1, 4), seq_len=i32(1),
                slopes=torch.zeros(4, device=dev), prefix_len=i32(1), lse=torch.zeros(1, 4, device=dev),
                ws=torch.zeros(1 << 20, dtype=torch.uint8, device=dev))
    calls = {
        "tables": (cache.bind_tables, dict(pages=i32(8), past_len=i32(1), new_len=i32(1)), dict(tables=t)),
        "write": (cache.bind_write, dict(q=half(1, 4, 64), k=half(1, 2, 64), v=half(1, 2, 64), q_out=half(1, 4, 64),
                                         position=i32(1), k_slots=i32(1).long(), v_slots=i32(1).long(),
                                         q_weight=half(64), k_weight=half(64)), dict(norm=True)),
        "decode": (cache.bind_decode, attn, {}),
        "prefill": (cache.bind_prefill, dict(attn, q_offsets=i32(2)), {}),
    }
    for what, (bind, tensors, more) in calls.items():
        bind(**tensors, **more)
        for name, x in tensors.items():
            with pytest.raises(ValueError, match=f"{name}: expected a tensor on"):
                bind(**{**tensors, name: x.cpu()}, **more)
    host = rt.Rope(64, device="cpu")
    with pytest.raises(ValueError, match="rope.turns: expected a tensor on"):
        cache.bind_write(**calls["write"][1], rope=host)
    with pytest.raises(ValueError, match="contiguous"):
        cache.bind_decode(**{**attn, "ws": torch.zeros(1 << 20, 2, dtype=torch.uint8, device=dev)[:, 0]})
    # a workspace of another type counts by its bytes
    cache.bind_decode(**{**attn, "ws": torch.zeros(1 << 18, dtype=torch.int32, device=dev)})()
    torch.cuda.synchronize()
