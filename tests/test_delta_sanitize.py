"""The host plan of the delta's gradients built with g++ under AddressSanitizer and
UndefinedBehaviorSanitizer and driven by tests/delta_sanitize.cpp.  CPU only."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "lora_adapter_pool_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_delta_plan_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "delta_sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
           "-I" + os.path.join(os.path.dirname(HERE), "include"), "-I" + CSRC,
           os.path.join(CSRC, "lora_host.cpp"), os.path.join(CSRC, "lora_delta_plan.cpp"),
           os.path.join(HERE, "delta_sanitize.cpp"), "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe, "400"], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True,
                       timeout=300, env=env)
    assert r.returncode == 0, r.stdout
    assert "0 failed checks" in r.stdout
