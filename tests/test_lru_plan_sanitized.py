"""The recurrence's host-side plan and the rotary frequencies (pure C++) built
with g++ under AddressSanitizer and UndefinedBehaviorSanitizer and run against
randomised batches and scalings (tests/native/lru_plan_fuzz.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_rnn_gated_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_lru_plan_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "lru_plan_fuzz")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "gdn_plan.cpp"), os.path.join(CSRC, "gdn_rope.cpp"),
           os.path.join(ROOT, "tests", "native", "lru_plan_fuzz.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "lru_plan_fuzz: ok" in r.stdout
