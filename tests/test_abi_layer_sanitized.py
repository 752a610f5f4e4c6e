"""The entry points of the operators around a layer's Linears built for the host with AddressSanitizer and
UndefinedBehaviorSanitizer, every size argument swept up to INT64_MAX singly and in pairs (tests/abi_layer_sanitize.cpp):
an overflowing size product in a check is a sanitizer report, and what passes the checks must satisfy the launchers'
assumptions."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "fp8_fine_grained_fp8bq_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"), reason="needs g++ and the HIP headers")
def test_entry_points_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "abi_layer_san")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
           os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "api_layer.cpp"), os.path.join(HERE, "abi_layer_sanitize.cpp"),
           "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "asan" in build.stderr.lower() and "cannot find" in build.stderr.lower():
        pytest.skip("sanitizer runtimes not installed: " + build.stderr[-300:])
    assert build.returncode == 0, build.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0", UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    print(res.stdout, res.stderr[-3000:])
    assert res.returncode == 0, res.stdout + res.stderr[-3000:]
