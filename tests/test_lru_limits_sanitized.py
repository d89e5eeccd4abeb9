"""The sizes that the gated linear recurrence takes and how it groups many sequences: its host-side plan (pure
C++) built with g++ under AddressSanitizer and UndefinedBehaviorSanitizer and run
against randomised sizes and batches (tests/native/lru_limits_fuzz.cpp, lru_units_fuzz.cpp)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_rnn_gated_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
@pytest.mark.parametrize("name", ["lru_limits_fuzz", "lru_units_fuzz"])
def test_lru_limits_under_asan_ubsan(tmp_path, name):
    exe = str(tmp_path / name)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "gdn_plan.cpp"),
           os.path.join(ROOT, "tests", "native", name + ".cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert name + ": ok" in r.stdout
