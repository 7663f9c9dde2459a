"""The cache in 4 bits without a GPU: refusals (before any launch), sizes, and the references the
GPU tests are held to, with mistakes planted in them."""

import ctypes
import math

import numpy as np
import pytest
import torch

import kv4_util as four
import kv_util as util
from heterogeneous_lora_amd import _lib, runtime
from test_kv_host import BAD_LENGTHS, BAD_PAGES, DEV, attn, kv, qkv, r, refused

# (2 heads of 64: 2 x (32 + 2) bytes of a token, in whole 16s 80; 3 tokens are 240 of 512)
FOUR = dict(tokens_per_page=3)
PAGES = [x for x in BAD_PAGES if "fit" not in x[1]] + [
    (dict(page_elems=112), "3 tokens of 80 bytes"), (dict(tokens_per_page=7), "7 tokens of 80 bytes"),
    (dict(n_kv_heads=1025), "n_kv_heads")]
LENGTHS = [x for x in BAD_LENGTHS if "max_blocks" not in x[1]] + [(dict(max_blocks=-1), "max_blocks"),
                                                                 (dict(max_blocks=(1 << 30) // 3 + 1), "max_blocks")]


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _lib.load()


def kv4(**over):
    return kv(**{**FOUR, **over})


def rows(**over):
    f = dict(n_tokens=4, k=DEV, k_token_stride=128, k_head_stride=64, v=DEV, v_token_stride=128, v_head_stride=64,
             k_slots=DEV, v_slots=DEV)
    f.update(over)
    return _lib.KVRows(**f)


def _workspace(k, a, n=0):
    b = ctypes.c_int64()
    rc = _lib.load().slora_attn4_workspace_size(r(k), r(a), n, r(b))
    return rc, b.value


@pytest.mark.parametrize("over,match", PAGES + LENGTHS[:3])
def test_write_and_read_refuse_geometry(over, match):
    refused(_lib.bind_kv4_write, kv4(**over), qkv(), 0, match=match)
    refused(_lib.bind_kv4_read, kv4(**over), rows(), 0, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(n_tokens=-1), "n_tokens"), (dict(n_q_heads=0), "n_q_heads"), (dict(rotary_dim=72), "rotary_dim"),
    (dict(eps=math.nan), "eps"), (dict(q=None), "q must"), (dict(q_out=DEV + 2), "q_out"), (dict(k=None), "together"),
    (dict(v_head_stride=12), "v strides"), (dict(k_slots=None), "k_slots"), (dict(position=None), "position"),
    (dict(turns=None), "turns"), (dict(k_weight=DEV + 4), "weights"), (dict(q_out=DEV, out_head_stride=128), "other strides")])
def test_write_refuses_arguments(over, match):
    refused(_lib.bind_kv4_write, kv4(), qkv(**over), 0, match=match)


@pytest.mark.parametrize("over,match", [
    (dict(n_tokens=-1), "n_tokens"), (dict(k=DEV + 2), "k must"), (dict(v=DEV + 8), "v must"),
    (dict(k_token_stride=100), "k strides"), (dict(v_head_stride=63), "v strides"), (dict(k_slots=None), "k_slots"),
    (dict(v_slots=None), "v_slots")])
def test_read_refuses_arguments(over, match):
    refused(_lib.bind_kv4_read, kv4(), rows(**over), 0, match=match)


@pytest.mark.parametrize("over,match", LENGTHS + PAGES)
def test_attention_refuses_geometry(over, match):
    refused(_lib.bind_attn4_decode, kv4(**over), attn(), DEV, 1 << 40, 0, match=match)
    refused(_lib.bind_attn4_prefill, kv4(**over), attn(), DEV, 4, DEV, 1 << 40, 0, match=match)
    assert _workspace(kv4(**over), attn())[0] == _lib.E_INVALID


@pytest.mark.parametrize("over,match", [
    (dict(n_q_heads=3), "n_q_heads"), (dict(scale=math.nan), "scale"), (dict(softcap=-1.0), "softcap"),
    (dict(window=-1), "window"), (dict(seq_len=None), "seq_len"), (dict(k_table=None), "k_table"),
    (dict(v_table=None), "v_table"), (dict(q=None), "q must"), (dict(out=DEV + 6), "out must"),
    (dict(out_token_stride=100), "out strides")])
def test_attention_refuses_arguments(over, match):
    refused(_lib.bind_attn4_decode, kv4(), attn(**over), DEV, 1 << 40, 0, match=match)
    refused(_lib.bind_attn4_prefill, kv4(), attn(**over), DEV, 4, DEV, 1 << 40, 0, match=match)


@pytest.mark.parametrize("n_requests,max_blocks", [(3, 8), (3, 200000)])  # few keys, many
def test_attention_refuses_workspaces_and_offsets(n_requests, max_blocks):
    k = kv4(n_requests=n_requests, max_blocks=max_blocks)
    rc, need = _workspace(k, attn())
    assert rc == _lib.OK and need >= 256
    refused(_lib.bind_attn4_decode, k, attn(), None, need, 0, match="ws must")
    refused(_lib.bind_attn4_decode, k, attn(), DEV + 16, need, 0, match="ws must")
    refused(_lib.bind_attn4_decode, k, attn(), DEV, need - 1, 0, match="smaller than")
    refused(_lib.bind_attn4_prefill, k, attn(), None, 4, DEV, 1 << 40, 0, match="q_offsets")
    refused(_lib.bind_attn4_prefill, k, attn(), DEV, -1, DEV, 1 << 40, 0, match="n_tokens")
    for n in (4, 20000):  # (20000 tokens: read back first, where they fit)
        rc, need = _workspace(k, attn(), n)
        assert rc == _lib.OK
        refused(_lib.bind_attn4_prefill, k, attn(), DEV, n, DEV, need - 1, 0, match="smaller than")
    assert _workspace(k, attn(), -1)[0] == _lib.E_INVALID


def test_calls_with_nothing_to_do_launch_nothing():
    _lib.bind_kv4_write(kv4(), qkv(n_tokens=0, q=None, k=None, v=None), 0)()
    _lib.bind_kv4_read(kv4(), rows(n_tokens=0, k=None, v=None), 0)()
    _lib.bind_kv4_read(kv4(), rows(k=None, v=None, k_slots=None, v_slots=None), 0)()
    _lib.bind_attn4_decode(kv4(n_requests=0), attn(), None, 0, 0)()
    _lib.bind_attn4_prefill(kv4(n_requests=0), attn(), None, 4, None, 0, 0)()
    _lib.bind_attn4_prefill(kv4(), attn(), None, 0, None, 0, 0)()


def test_null_arguments():
    lib, k, b = _lib.load(), kv4(), ctypes.c_int64()
    null = ctypes.c_void_p(None)
    for rc in (lib.slora_kv4_token_bytes(2, 64, None), lib.slora_kv4_write(null, r(qkv()), null),
               lib.slora_kv4_write(r(k), null, null), lib.slora_kv4_read(r(k), null, null),
               lib.slora_kv4_read(null, r(rows()), null), lib.slora_attn4_workspace_size(r(k), null, 0, r(b)),
               lib.slora_attn4_workspace_size(r(k), r(attn()), 0, None), lib.slora_attn4_decode(r(k), null, null, 0, null),
               lib.slora_attn4_prefill(null, r(attn()), null, 1, null, 0, null)):
        assert rc == _lib.E_INVALID


@pytest.mark.parametrize("hk", [1, 2, 3, 8, 40, 1024])
def test_token_bytes(hk):
    for d in range(8, 257, 8):
        assert _lib.kv4_token_bytes(hk, d) == four.layout(hk, d)[2]
    for bad in (0, 4, 12, 264):
        with pytest.raises(_lib.SloraError, match="head_dim"):
            _lib.kv4_token_bytes(hk, bad)


def test_workspaces_grow_with_what_is_asked():
    """Enough for every window; read-back blocks are asked for where they are used, never above 1 GiB."""
    sizes = [_workspace(kv4(n_requests=64, max_blocks=20000), attn(window=w))[1] for w in (0, 1, 5000, 1 << 30)]
    assert len(set(sizes)) == 1
    short, long = (_workspace(kv4(n_requests=1, max_blocks=2000), attn(), n)[1] for n in (2000, 3000))
    # (2 query heads a KV head: 4096 rows from 2048 tokens on; 6000 tokens are 94 blocks of 64)
    assert long - short >= 94 * 64 * 2 * 64 * 4
    assert _workspace(kv4(n_requests=64, max_blocks=1 << 28, tokens_per_page=1), attn(), 1 << 20)[1] < 1 << 30


# ---------------------------------------------------------------- KVCache

def test_cache_refuses_bits():
    for bits in (0, 8, 32, None):
        with pytest.raises(ValueError, match="bit"):
            runtime.KVCache(None, 4, bits=bits)


def test_read_is_of_4_bits():
    x = torch.zeros(4, 1, 8, dtype=torch.float16)
    at = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="bit"):
        runtime.KVCache(None, 4, page_elems=8).bind_read(x, x, at, at)


def test_host_tensors_are_refused():
    cache = runtime.KVCache(None, 4, page_elems=64, n_kv_heads=2, head_dim=64, bits=4)
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    at = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU|device|cuda"):
        cache.bind_read(x, x, at, at)
    with pytest.raises(ValueError, match="expected"):
        cache.bind_read(x.float(), None, at, None)


# ---------------------------------------------------------------- the references

def test_held_by_hand():
    """Groups worked out on paper: ties go to the even level, steps to the even of two."""
    def one(*x):
        return four.held(torch.tensor([list(x) + [0.0] * (32 - len(x))], dtype=torch.float64))
    code, step = one(6.0, 5.0, -2.5, 0.25, 0.75, 1.25, -1.75, 3.5, 0.2500001, -0.0)
    assert int(step) == 15 * 8  # 1.0
    # 5 lies between 4 and 6: codes 6 and 7; 2.5: 2 and 3 (4, 5); .25: 0 and .5 (0, 1); .75 (1, 2); 1.25 (2, 3);
    # 1.75 (3, 4); 3.5 (5, 6)
    assert code[0, 0, :10].tolist() == [7, 6, 12, 0, 2, 2, 12, 6, 1, 8]
    assert int(one(6 * 1.0625)[1]) == 120 and int(one(6 * 1.1875)[1]) == 122  # halves to the even step
    assert int(one(65504.0)[1]) == 226 and int(one(1e300)[1]) == 226  # 10240, and 6 of it in f16
    assert int(one(6 * 2.0 ** -17)[1]) == 1 and int(one(6 * 2.0 ** -18)[1]) == 0  # smallest step; half of it
    for bad in (math.inf, -math.inf, math.nan):
        code, step = one(1.0, bad)
        assert int(step) == 255 and not bool(code.any())


@pytest.mark.parametrize("d", [8, 32, 40, 128, 256])
def test_values_are_close_and_exact_in_both_types(d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(50, d, generator=g, dtype=torch.float64) * torch.logspace(-3, 3, 50, dtype=torch.float64)[:, None]
    code, step = four.held(x)
    v = four.values(code, step, d)
    for t in (torch.float16, torch.bfloat16):
        assert torch.equal(v.to(t).double(), v)
    size = four.STEPS[step].repeat_interleave(32, -1)[:, :d]
    # Levels are at most 2 apart, so half of that times the step; the largest magnitude is at most 6 / (1 - 1/17)
    # steps (a step is at most half of an eighth too small: 8.5 for 8 of 8ths)
    assert bool(((v - x).abs() <= size * (1 + 6.0 / 16)).all())


def test_bytes_of_a_token():
    code = torch.arange(2 * 2 * 32).reshape(1, 2, 2, 32) % 16
    step = torch.tensor([[[3, 4], [5, 6]]])
    raw = four.token_bytes(code, step, 2)[0].tolist()
    assert len(raw) == 80 and raw[64:68] == [3, 4, 5, 6] and raw[68:] == [-1] * 12
    # dims 32 c + 8 g .. + 7 of a head at word 2 g + c: c 1, g 1 (dims 40 ..) are word 3
    dims = [int(x) for x in code[0, 0].flatten()[40:48]]
    assert raw[12:16] == [dims[0] | dims[1] << 4, dims[2] | dims[3] << 4, dims[4] | dims[5] << 4, dims[6] | dims[7] << 4]


@pytest.mark.parametrize("mistake", ["step", "level", "head", "last key", "first key", "scale", "cap", "weights"])
def test_planted_mistakes_pass_the_bound(mistake):
    """What attention must not do is further off than the bound."""
    rng = np.random.default_rng(7)
    lens = [90, 200]
    make = lambda: four.Cache(np.random.default_rng(7), lens, dtype="f16", hk=2, d=64, tpp=3)
    c = make()
    q = (torch.from_numpy(rng.standard_normal((2, 4, 64))) * 1.5).half()
    at = [(0, 89), (1, 199)]
    kw = dict(scale=0.125, cap=20.0, window=100)
    ref = four.attention(c, q, at, **kw)
    bound = four.bound(ref, "f16", True)
    other = make()
    if mistake == "step":
        other.v = [v * (1 + 2.0 ** -4) for v in other.v]
    elif mistake == "level":
        k = other.k[0]
        k[50, 0, 7] += 0.5
        q2 = q
    elif mistake == "head":
        q = q[:, [0, 2, 1, 3]]
    elif mistake == "last key":
        at = [(0, 88), (1, 198)]
    elif mistake == "first key":
        kw["window"] = 99
    elif mistake == "scale":
        kw["scale"] = 0.126
    elif mistake == "cap":
        kw["cap"] = 0.0
    wrong = four.attention(other, q, at, rounded=torch.float8_e4m3fn if mistake == "weights" else None, **kw)
    assert bool(((wrong.out - ref.out).abs() > bound).any()), mistake
    assert bool(((ref.out.half().double() - ref.out).abs() <= bound).all())
