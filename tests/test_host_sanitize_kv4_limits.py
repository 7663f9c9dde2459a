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
