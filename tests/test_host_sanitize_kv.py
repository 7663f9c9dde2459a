"""The host code of the KV cache and attention calls under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/host_sanitize/kv_driver.cpp): argument checks, rotary
frequencies, magic divisors, and whether every counter and partial result of every shape of
call lies inside the workspace. No GPU is used."""

import os
import re
import subprocess

import pytest

import test_host_sanitize as base

# compiled into this driver; the others into test_host_sanitize's
HERE = ["kv.cpp"]


def test_every_host_source_is_sanitized():
    from heterogeneous_lora_amd import build
    assert sorted(build.HOST_SRCS) == sorted(base.HOST_SRCS + HERE)


@pytest.mark.skipif(not os.path.exists(base.CXX), reason="ROCm clang++ not found")
def test_kv_host_logic_under_sanitizers(tmp_path):
    csrc = os.path.join(base.ROOT, "heterogeneous_lora_amd", "csrc")
    inc = [f"-I{os.path.join(base.ROOT, 'include')}", f"-I{csrc}", f"-I{base.ROCM}/include", "-D__HIP_PLATFORM_AMD__=1"]
    srcs = [os.path.join(csrc, s) for s in HERE] + [os.path.join(base.ROOT, "tests", "host_sanitize", "kv_driver.cpp")]
    exe = str(tmp_path / "kv_driver")
    base._run([base.CXX, "-O1", "-g", "-std=c++17", *base.SAN, *inc, "-o", exe, *srcs])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    p = subprocess.run([exe, "120"], capture_output=True, text=True, env=env, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr[-4000:]
    assert "AddressSanitizer" not in p.stderr and "runtime error" not in p.stderr, p.stderr[-4000:]
    m = re.search(r"(\d+) calls, (\d+) refusals, (\d+) cut rows, (\d+) counters of (\d+) at most; 0 failed checks", p.stdout)
    assert m, p.stdout
    calls, refusals, cut, most, room = map(int, m.groups())
    assert calls > 1000 and refusals > 1000 and cut > 1000 and 256 < most <= room, p.stdout
