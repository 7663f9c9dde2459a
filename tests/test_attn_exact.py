"""The bounds of attn_exact on the CPU: weights rounded once to the storage type break the
bound that the two-part weights of the decode kernel are held to."""

import pytest
import torch

import attn_exact as ax
import kv_util as ku
from test_gpu_attention_weights import DECODE, LOST, decode_case


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("name", sorted(set(DECODE) - {"cut"}))  # (there f16's floor, times the keys, is above a rounding)
def test_bound_notices_weights_rounded_once(name, dtype):
    c, q, rows, scale = decode_case(name, dtype)
    ref = ax.attention(c, q, rows, scale=scale)
    b = ax.bound(ref, dtype, *LOST[dtype])
    ku.check(ref.out.to(ku.TORCH[dtype]), ref.out, b, "rounded result")
    once = ax.attention(c, q, rows, scale=scale, rounded=ku.TORCH[dtype])
    with pytest.raises(AssertionError, match="times the bound"):
        ku.check(once.out.to(ku.TORCH[dtype]), ref.out, b, "rounded weights")
    assert torch.isfinite(b).all()
