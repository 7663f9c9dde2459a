"""Attention whose keys are cut into chunks, waves that take heads of their own, workspaces
that calls share: against the references of kv_util."""

import numpy as np
import pytest
import torch

import kv_util as ku
from test_gpu_kv import _attn, _check_attn, _offsets, rt  # noqa: F401

pytestmark = pytest.mark.gpu
T = ku.TORCH

DECODE = {
    # enough requests for a head to each wave: 4 heads, 2 and 1 to a workgroup
    "four heads": dict(lens=[i % 9 for i in range(512)], hk=8, group=1, d=64),
    "two heads": dict(lens=[i % 7 for i in range(350)], hk=6, group=2, d=40, tpp=2),
    "one head": dict(lens=[i % 5 for i in range(220)], hk=5, group=1, d=128),
    "four heads, one long": dict(lens=[3] * 256 + [1900, 0, 77] + [2] * 260, hk=8, group=1, d=64, tpp=4),
    "more rows than 16": dict(lens=[2, 900], hk=4, group=20, d=64),
    "long, odd heads": dict(lens=[2000, 1, 1300], hk=3, group=2, d=72, tpp=5),
    "long, wide heads": dict(lens=[1500], hk=2, group=3, d=256),
    "long, window": dict(lens=[4000, 3000], hk=1, group=2, d=96, tpp=3, window=2000, prefix=[300, 40], cap=25.0, slopes=True),
}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(DECODE))
def test_decode(rt, name, dtype):  # noqa: F811
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, name, DECODE[name], dtype)
    cache, kt, vt = c.to_gpu()
    cache.decode(q.cuda(), out, kt, vt, seq, **dev)
    _check_attn(f"decode {name} {dtype}", c, q, rows, ref, out, lse)
    again = torch.zeros_like(out)  # whichever workgroup joins, the same bits
    cache.decode(q.cuda(), again, kt, vt, seq, **dev)
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(out))


PREFILL = {
    "one row": dict(lens=[3000], new=[1], hk=2, group=1, d=64),
    "rows of two tiles": dict(lens=[2600], new=[70], hk=1, group=2, d=128, tpp=4),
    "uneven requests": dict(lens=[2900, 20, 700, 0, 1400], new=[3, 20, 40, 0, 1], hk=2, group=2, d=64, tpp=3),
    "heads of 96": dict(lens=[1800], new=[9], hk=1, group=4, d=96),
    "heads of 192": dict(lens=[1700], new=[5], hk=1, group=2, d=192, tpp=2),
    "heads of 256": dict(lens=[1700], new=[5], hk=1, group=1, d=256),
    "window": dict(lens=[3000, 1500], new=[20, 30], hk=1, group=2, d=64, window=1200, prefix=[70, 1400]),
    "everything": dict(lens=[2500], new=[40], hk=1, group=4, d=80, tpp=4, cap=20.0, slopes=True, window=1500, prefix=[130]),
    "many requests": dict(lens=[700 if i % 30 == 0 else i % 4 for i in range(150)], new=[i % 4 and 1 for i in range(150)], hk=1, group=1, d=64),
}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(PREFILL))
def test_prefill(rt, name, dtype):  # noqa: F811
    spec = PREFILL[name]
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, name, spec, dtype, spec["new"])
    cache, kt, vt = c.to_gpu()
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets(spec["new"]), **dev)
    _check_attn(f"prefill {name} {dtype}", c, q, rows, ref, out, lse)
    again = torch.zeros_like(out)
    cache.prefill(q.cuda(), again, kt, vt, seq, _offsets(spec["new"]), **dev)
    assert torch.equal(again, out)


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_of_zero_and_below(rt, scale):  # noqa: F811
    spec = dict(lens=[90, 40], new=[50, 40], hk=1, group=2, d=64)
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, "", spec, "f16", spec["new"])
    ref["scale"] = dev["scale"] = scale
    cache, kt, vt = c.to_gpu()
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets(spec["new"]), **dev)
    _check_attn(f"prefill, scale {scale}", c, q, rows, ref, out, lse)
    last = q[[49, 89]]
    got, got_lse = torch.empty(2, 2, 64, dtype=torch.float16, device="cuda"), torch.empty(2, 2, device="cuda")
    cache.decode(last.cuda(), got, kt, vt, seq, scale=scale, lse=got_lse)
    _check_attn(f"decode, scale {scale}", c, last, [(0, 89), (1, 39)], ref, got, got_lse)


def test_infinities_in_cut_rows(rt):  # noqa: F811
    """A chunk's infinities and NaN reach the rows that see them, and only those."""
    spec = dict(lens=[2000], new=[40], hk=1, group=2, d=64, window=1300)
    c, q, rows, ref, out, lse, dev, seq = _attn(rt, "", spec, "bf16", spec["new"])
    c.set_v(0, 680, float("inf"), dim=5)   # leaves the window within the rows
    c.set_v(0, 1000, float("-inf"), dim=9)
    c.set_v(0, 1980, float("nan"), dim=63)  # new: later rows alone
    cache, kt, vt = c.to_gpu()
    cache.prefill(q.cuda(), out, kt, vt, seq, _offsets([40]), **dev)
    want, bound, _ = ku.attention(c, q, rows, **ref)
    assert torch.isinf(want[0, :, 5]).all() and torch.isfinite(want[-1, :, 5]).all()
    assert torch.isfinite(want[0, :, 63]).all() and torch.isnan(want[-1, :, 63]).all()
    ku.check(out, want, bound, "prefill")
    c.set_v(0, 1980, 0.5, dim=63)
    cache, kt, vt = c.to_gpu()
    got = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache.decode(q[-1:].cuda(), got, kt, vt, seq, scale=ref["scale"])
    want, bound, _ = ku.attention(c, q[-1:], [(0, 1999)], scale=ref["scale"])
    assert torch.isinf(want[0, :, 5]).all() and torch.isinf(want[0, :, 9]).all()
    ku.check(got, want, bound, "decode")


def test_calls_share_a_workspace(rt):  # noqa: F811
    """Calls of several shapes, one after the other in one workspace, equal calls with their own."""
    from heterogeneous_lora_amd import _lib
    cases = []
    for lens, new, hk, group, d in (([2500, 9], [3, 9], 2, 2, 64), ([1600], [30], 1, 4, 128), ([800] * 5, [1] * 5, 4, 1, 96)):
        spec = dict(lens=lens, new=new, hk=hk, group=group, d=d)
        c, q, rows, ref, out, lse, dev, seq = _attn(rt, "", spec, "f16", new)
        cases.append((c.to_gpu(), q.cuda(), seq, new, dev["scale"]))
    ws = torch.zeros(96 << 20, dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for (cache, kt, vt), q, seq, new, scale in cases:
            last = q[(_offsets(new)[1:] - 1).long()].contiguous()
            for w in (None, ws):
                a, b = torch.empty_like(q), torch.empty_like(last)
                cache.prefill(q, a, kt, vt, seq, _offsets(new), scale=scale, ws=w)
                cache.decode(last, b, kt, vt, seq, scale=scale, ws=w)
                if w is None:
                    want = a, b
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert int(ws[:10240].view(torch.int32).abs().max()) == 0
