"""The state space layer's host code under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU, at the largest sizes that it takes
(tests/layer_spans_sanitize.cpp): the extents of buffers do not overflow on their way
to 64 bits."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_spans_of_the_largest_sizes(tmp_path):
    exe = str(tmp_path / "layer_spans_sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(ROOT, "recurrent_state_update_amd", "csrc"),
           "-x", "c++", os.path.join(HERE, "layer_spans_sanitize.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    report = r.stdout + r.stderr
    assert r.returncode == 0, report
    assert "ERROR:" not in report and "runtime error" not in report, report
    assert "layer span checks passed" in r.stdout
