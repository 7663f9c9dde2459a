"""The host code of the cache in 4 bits under AddressSanitizer and UndefinedBehaviorSanitizer
(tests/host_sanitize/kv4_driver.cpp): argument checks, and whether every partial result, cut and
block read back has its own place inside the workspace. No GPU is used."""

import os
import re
import subprocess

import pytest

import test_host_sanitize as base


@pytest.mark.skipif(not os.path.exists(base.CXX), reason="ROCm clang++ not found")
def test_kv4_host_logic_under_sanitizers(tmp_path):
    csrc = os.path.join(base.ROOT, "heterogeneous_lora_amd", "csrc")
    inc = [f"-I{os.path.join(base.ROOT, 'include')}", f"-I{csrc}", f"-I{base.ROCM}/include", "-D__HIP_PLATFORM_AMD__=1"]
    exe = str(tmp_path / "kv4_driver")
    base._run([base.CXX, "-O1", "-g", "-std=c++17", *base.SAN, *inc, "-o", exe,
               os.path.join(base.ROOT, "tests", "host_sanitize", "kv4_driver.cpp")])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe, "100"], capture_output=True, text=True, env=env, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr[-4000:]
    assert "AddressSanitizer" not in p.stderr and "runtime error" not in p.stderr, p.stderr[-4000:]
    m = re.search(r"(\d+) few, (\d+) spans, (\d+) straight, (\d+) back, (\d+) cut, (\d+) refusals; 0 failed checks", p.stdout)
    assert m, p.stdout
    assert all(int(x) > 100 for x in m.groups()), p.stdout
