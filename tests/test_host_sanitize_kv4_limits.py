"""Sizes of workspaces at the largest numbers the calls accept, under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/host_sanitize/kv4_limits_driver.cpp). No GPU is used."""

import os
import subprocess

import pytest

import test_host_sanitize as base


def run_driver(tmp_path, name):
    csrc = os.path.join(base.ROOT, "heterogeneous_lora_amd", "csrc")
    inc = [f"-I{os.path.join(base.ROOT, 'include')}", f"-I{csrc}", f"-I{base.ROCM}/include", "-D__HIP_PLATFORM_AMD__=1"]
    exe = str(tmp_path / name)
    base._run([base.CXX, "-O1", "-g", "-std=c++17", *base.SAN, *inc, "-o", exe,
               os.path.join(base.ROOT, "tests", "host_sanitize", f"{name}.cpp")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert "AddressSanitizer" not in p.stderr and "runtime error" not in p.stderr, p.stderr[-4000:]
    assert p.returncode == 0, p.stdout + p.stderr[-4000:]
    return p.stdout


@pytest.mark.skipif(not os.path.exists(base.CXX), reason="ROCm clang++ not found")
def test_sizes_at_the_limits(tmp_path):
    out = run_driver(tmp_path, "kv4_limits_driver")
    assert out == "1536 sizes; 0 failed checks\n", out


def test_a_wide_table_does_not_ask_for_its_keys():
    """A prompt's workspace over 4 bits beside the one over 16: by q and out, not by the table."""
    from heterogeneous_lora_amd import _lib
    a = _lib.Attn(n_q_heads=32)
    extra = {}
    for tokens in (1023, 1024, 1025, 16000):
        for table in (1040, 4096, 16000, 16640, 131072, 262000, 263000, 1 << 20):
            sizes = []
            for bits in (16, 4):
                P = 8 * 128 if bits == 16 else _lib.kv4_token_bytes(8, 128) // 2
                kv = _lib.KV(1 << 20, 1 << 20, P, _lib.DTYPES["bf16"], 8, 128, 1, 1, table)
                sizes.append((_lib.attn_workspace_size if bits == 16 else _lib.attn4_workspace_size)(kv, a, tokens))
            extra[tokens, table] = sizes[1] - sizes[0]
            assert extra[tokens, table] <= 4 * (2 * tokens * 32 * 128 * 2) + table // 64 * 8 + 1024
    assert extra[1024, 4096] == 4096 // 64 * 8 + 4096 * 8 * 128 * 4  # read back: both tables, K and V
    assert extra[1023, 4096] == extra[1024, 131072] == extra[1024, 1 << 20] == 0
