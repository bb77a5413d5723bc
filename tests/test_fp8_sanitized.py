"""The argument checks of the 8-bit entry points under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only, tests/native/fp8_sanitize.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_fp8_checks_under_asan_ubsan(tmp_path):
    exe = tmp_path / "fp8_sanitize"
    build = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
             "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-I", os.path.join(ROOT, "include"),
             os.path.join(ROOT, "rotated_bit_amd", "csrc", "validate.cpp"),
             os.path.join(ROOT, "tests", "native", "fp8_sanitize.cpp"), "-o", str(exe)]
    b = subprocess.run(build, capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    env.pop("LD_PRELOAD", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "all checks passed" in r.stdout and "runtime error" not in r.stderr
