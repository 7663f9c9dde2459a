"""KV cache and attention entry points without a GPU: refusals (before any launch) and the
rotary frequencies against their formulas."""

import ctypes
import math

import numpy as np
import pytest

from heterogeneous_lora_amd import _lib

DEV = 0x7F0000000000  # never dereferenced by host code


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _lib.load()


def kv(**over):
    f = dict(pool=DEV, n_pages=64, page_elems=256, dtype=_lib.F16, n_kv_heads=2, head_dim=64,
             tokens_per_page=2, n_requests=3, max_blocks=8)
    f.update(over)
    return _lib.KV(**f)


def step(**over):
    f = dict(n_planes=2, append=0, pages=DEV, n_page_ids=48, past_len=DEV, new_len=DEV, n_tokens=4, tables=DEV,
             seq_len=DEV, q_offsets=DEV, token_request=DEV, position=DEV, slots=DEV)
    f.update(over)
    return _lib.KVStep(**f)


def qkv(**over):
    f = dict(n_tokens=4, n_q_heads=4, q=DEV, q_token_stride=256, q_head_stride=64, k=DEV, k_token_stride=128,
             k_head_stride=64, v=DEV, v_token_stride=128, v_head_stride=64, q_out=DEV + 4096,
             out_token_stride=256, out_head_stride=64, position=DEV, k_slots=DEV, v_slots=DEV, turns=DEV,
             rotary_dim=64, interleaved=0, cos_sin_scale=1.0, norm=1, eps=1e-6, q_weight=DEV, k_weight=DEV)
    f.update(over)
    return _lib.QKV(**f)


def attn(**over):
    f = dict(n_q_heads=4, scale=0.125, softcap=0.0, window=0, slopes=None, prefix_len=None, k_table=DEV,
             v_table=DEV, seq_len=DEV, q=DEV, q_token_stride=256, q_head_stride=64, out=DEV + 4096,
             out_token_stride=256, out_head_stride=64, lse=None)
    f.update(over)
    return _lib.Attn(**f)


def refused(bind, *args, match):
    with pytest.raises(_lib.SloraError, match=match) as e:
        bind(*args)()
    assert e.value.code == _lib.E_INVALID


def r(x):
    return ctypes.byref(x)


BAD_LENGTHS = [(dict(n_pages=-1), "n_pages"), (dict(n_pages=1 << 31), "n_pages"),
               (dict(tokens_per_page=0), "tokens_per_page"), (dict(n_requests=-1), "n_requests"),
               (dict(n_requests=16385), "n_requests"), (dict(max_blocks=-1), "max_blocks"),
               (dict(max_blocks=1 << 30), "max_blocks")]
BAD_PAGES = [(dict(pool=None), "pool"), (dict(pool=DEV + 8), "pool"), (dict(dtype=2), "dtype"),
             (dict(page_elems=252), "page_elems"), (dict(page_elems=0), "page_elems"),
             (dict(head_dim=60), "head_dim"), (dict(head_dim=264), "head_dim"), (dict(head_dim=0), "head_dim"),
             (dict(n_kv_heads=0), "n_kv_heads"), (dict(page_elems=248), "do not fit")]


@pytest.mark.parametrize("over,match", BAD_LENGTHS)
def test_tables_refuses_geometry(over, match):
    refused(_lib.bind_kv_tables, kv(**over), step(), 0, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(n_planes=0), "n_planes"), (dict(n_planes=4097), "n_planes"), (dict(n_tokens=-1), "n_tokens"),
    (dict(n_page_ids=-1), "n_page_ids"), (dict(pages=None), "pages"), (dict(tables=None), "tables"),
    (dict(q_offsets=None), "length array"), (dict(past_len=None), "length array"), (dict(new_len=None), "length array"),
    (dict(seq_len=None), "length array"), (dict(slots=None), "token array"), (dict(position=None), "token array"),
    (dict(token_request=None), "token array")])
def test_tables_refuses_arguments(over, match):
    refused(_lib.bind_kv_tables, kv(), step(**over), 0, match=match)


@pytest.mark.parametrize("over,match", BAD_PAGES)
def test_write_refuses_geometry(over, match):
    refused(_lib.bind_kv_write, kv(**over), qkv(), 0, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(n_tokens=-1), "n_tokens"), (dict(n_q_heads=0), "n_q_heads"), (dict(rotary_dim=72), "rotary_dim"),
    (dict(rotary_dim=20), "rotary_dim"), (dict(rotary_dim=-8), "rotary_dim"), (dict(eps=-1.0), "eps"),
    (dict(eps=math.nan), "eps"), (dict(q=None), "q must"), (dict(q=DEV + 2), "q must"), (dict(q_out=None), "q_out"),
    (dict(q_token_stride=4), "q strides"), (dict(q_head_stride=63), "q strides"), (dict(k=None), "together"),
    (dict(v=None), "together"), (dict(k=DEV + 4), "k must"), (dict(v_head_stride=12), "v strides"),
    (dict(k_slots=None), "k_slots"), (dict(v_slots=None), "v_slots"), (dict(position=None), "position"),
    (dict(turns=None), "turns"), (dict(q_weight=DEV + 4), "weights"), (dict(q_out=DEV, out_head_stride=128), "other strides")])
def test_write_refuses_arguments(over, match):
    refused(_lib.bind_kv_write, kv(), qkv(**over), 0, match=match)


def _workspace(k, a, n=0):
    b = ctypes.c_int64()
    rc = _lib.load().slora_attn_workspace_size(r(k), r(a), n, r(b))
    return rc, b.value


@pytest.mark.parametrize("over,match", BAD_LENGTHS + BAD_PAGES)
def test_attention_refuses_geometry(over, match):
    refused(_lib.bind_attn_decode, kv(**over), attn(), DEV, 1 << 40, 0, match=match)
    refused(_lib.bind_attn_prefill, kv(**over), attn(), DEV, 4, DEV, 1 << 40, 0, match=match)
    assert _workspace(kv(**over), attn())[0] == _lib.E_INVALID


@pytest.mark.parametrize("over,match", [
    (dict(n_q_heads=3), "n_q_heads"), (dict(n_q_heads=0), "n_q_heads"), (dict(scale=math.inf), "scale"),
    (dict(scale=math.nan), "scale"), (dict(softcap=-1.0), "softcap"), (dict(softcap=math.inf), "softcap"),
    (dict(window=-1), "window"), (dict(seq_len=None), "seq_len"), (dict(k_table=None), "k_table"),
    (dict(v_table=None), "v_table"), (dict(q=None), "q must"), (dict(out=DEV + 6), "out must"),
    (dict(out_token_stride=100), "out strides")])
def test_attention_refuses_arguments(over, match):
    refused(_lib.bind_attn_decode, kv(), attn(**over), DEV, 1 << 40, 0, match=match)
    refused(_lib.bind_attn_prefill, kv(), attn(**over), DEV, 4, DEV, 1 << 40, 0, match=match)


def test_attention_refuses_workspaces_and_offsets():
    rc, need = _workspace(kv(), attn())
    assert rc == _lib.OK and need >= 256
    refused(_lib.bind_attn_decode, kv(), attn(), None, need, 0, match="ws must")
    refused(_lib.bind_attn_decode, kv(), attn(), DEV + 16, need, 0, match="ws must")
    refused(_lib.bind_attn_decode, kv(), attn(), DEV, need - 1, 0, match="smaller than")
    refused(_lib.bind_attn_prefill, kv(), attn(), None, 4, DEV, 1 << 40, 0, match="q_offsets")
    refused(_lib.bind_attn_prefill, kv(), attn(), DEV, -1, DEV, 1 << 40, 0, match="n_tokens")
    refused(_lib.bind_attn_prefill, kv(), attn(), DEV, 4, DEV, 0, 0, match="smaller than")
    assert _workspace(kv(), attn(), -1)[0] == _lib.E_INVALID


def test_calls_with_nothing_to_do_launch_nothing():
    _lib.bind_kv_write(kv(), qkv(n_tokens=0, q=None, k=None, v=None), 0)()
    _lib.bind_attn_decode(kv(n_requests=0), attn(q=None), None, 0, 0)()
    _lib.bind_attn_prefill(kv(n_requests=0), attn(), None, 4, None, 0, 0)()
    _lib.bind_attn_prefill(kv(), attn(), None, 0, None, 0, 0)()


def test_null_arguments():
    lib = _lib.load()
    assert lib.slora_kv_tables(None, r(step()), None) == _lib.E_INVALID
    assert lib.slora_kv_tables(r(kv()), None, None) == _lib.E_INVALID
    assert lib.slora_kv_write(r(kv()), None, None) == _lib.E_INVALID
    assert lib.slora_attn_decode(None, r(attn()), None, 0, None) == _lib.E_INVALID
    assert lib.slora_attn_prefill(r(kv()), None, None, 1, None, 0, None) == _lib.E_INVALID
    assert lib.slora_rope_turns(None, None) == _lib.E_INVALID


@pytest.mark.parametrize("d", [8, 64, 72, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands"])
def test_rope_turns(d, scaling):
    f, theta, n0, lo, hi = 8.0, 10000.0, 2048.0, 1.0, 4.0
    got = _lib.rope_turns(_lib.Rope(d, _lib.ROPE_SCALING[scaling], theta, f, n0, lo, hi))
    i = np.arange(d // 2)
    t = np.float64(theta * (f ** (d / (d - 2)) if scaling == "base" else 1.0)) ** (-2.0 * i / d) / (2 * np.pi)
    if scaling == "linear":
        t = t / f
    if scaling == "bands":
        keep = np.clip((t * n0 - lo) / (hi - lo), 0, 1)
        assert d < 64 or (keep[0] == 1 and keep[-1] == 0 and ((keep > 0) & (keep < 1)).any())
        t = t * (keep + (1 - keep) / f)
    np.testing.assert_allclose(got[:d // 2], t, rtol=1e-14)


@pytest.mark.parametrize("over", [dict(rotary_dim=4), dict(rotary_dim=12), dict(rotary_dim=264), dict(scaling=4),
                                  dict(theta=0.0), dict(theta=math.nan), dict(factor=-1.0),
                                  dict(scaling=3, low_turns=4.0), dict(scaling=3, original_len=0.0)])
def test_rope_refuses(over):
    f = dict(rotary_dim=64, scaling=0, theta=1e4, factor=2.0, original_len=2048.0, low_turns=1.0, high_turns=4.0)
    f.update(over)
    with pytest.raises(_lib.SloraError) as e:
        _lib.rope_turns(_lib.Rope(**f))
    assert e.value.code == _lib.E_INVALID
