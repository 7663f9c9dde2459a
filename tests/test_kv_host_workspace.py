"""Sizes of the attention calls' workspaces: what chunks need, and the refusal of less."""

import pytest

from heterogeneous_lora_amd import _lib
from test_kv_host import DEV, _workspace, attn, kv, refused


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _lib.load()


def test_prefill_needs_room_for_parts_only_where_tiles_are_cut():
    rc, least = _workspace(kv(), attn(), 4)  # 16 tokens at most: nothing to cut
    assert rc == _lib.OK
    long = dict(max_blocks=1 << 16)
    rc, few = _workspace(kv(**long), attn(), 4)
    # parts of one wave: 256 chunks past one a tile for each of 2 KV heads, twice, 33 KiB at most
    assert rc == _lib.OK and least < few <= least + 2 * 256 * 2 * 33 * 1024
    rc, many = _workspace(kv(**long), attn(), 1 << 16)  # tiles alone fill the device
    assert rc == _lib.OK and many == least
    refused(_lib.bind_attn_prefill, kv(**long), attn(), DEV, 4, DEV, few - 1, 0, match="smaller than")


def test_decode_needs_more_for_more_requests():
    sizes = []
    for n in (1, 3, 100, 2000, 16384):
        rc, b = _workspace(kv(n_requests=n), attn())
        assert rc == _lib.OK
        sizes.append(b)
    assert sizes == sorted(sizes) and len(set(sizes)) == len(sizes)
    refused(_lib.bind_attn_decode, kv(n_requests=2000), attn(), DEV, sizes[2], 0, match="smaller than")


def test_heads_of_any_number_fit_the_counters():
    """Counters: chunks aimed for times the workgroups that share a chunk, within the region's 2560."""
    for hk, group in ((1, 1), (1, 16384), (4, 4096), (7, 3), (1024, 16), (1021, 1), (6, 17)):
        k = kv(n_kv_heads=hk, head_dim=8, page_elems=16384, tokens_per_page=1, n_requests=5, max_blocks=1 << 20)
        a = attn(n_q_heads=hk * group)
        for n in (0, 1, 64):
            rc, b = _workspace(k, a, n)
            assert rc == _lib.OK and b >= 10240
