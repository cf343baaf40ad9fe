"""The host code behind include/moe_block.h under AddressSanitizer and UndefinedBehaviorSanitizer (CPU only).

abi.cpp and abi_block.cpp are built with g++ together with host-only stand-ins of the kernel launchers
(abi_host_stubs.cpp, block_host_stubs.cpp); a child Python process preloads the sanitizer runtime, points
the binding at that library and runs tests/test_block_cpu.py (refusals, zero tokens) and
tests/block_stub_checks.py (valid calls).  Any sanitizer report aborts the child and fails the test.
"""

import os
import subprocess
import sys

import pytest

from test_abi_sanitize import CSRC, ROCM, ROOT, _asan_runtime


@pytest.mark.timeout(600)
def test_block_host_code_under_asan_and_ubsan(tmp_path):
    asan = _asan_runtime()
    if asan is None or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime_api.h")):
        pytest.skip("g++ with libasan and the HIP headers are needed")
    lib = str(tmp_path / "libmoe_block_sanitized.so")
    tests = os.path.join(ROOT, "tests")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "abi.cpp"), os.path.join(CSRC, "abi_block.cpp"), os.path.join(tests, "abi_host_stubs.cpp"),
           os.path.join(tests, "block_host_stubs.cpp"), "-o", lib]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert res.returncode == 0, res.stdout
    runner = ("import sys; sys.path[:0] = [%r, %r]; import sparse_moe_expert_route_amd as m; m.lib_path = %r; "
              "import pytest; sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', '-p', 'no:xdist', %r, %r]))"
              % (ROOT, tests, lib, os.path.join(tests, "test_block_cpu.py"), os.path.join(tests, "block_stub_checks.py")))
    env = dict(os.environ)
    env["LD_PRELOAD"] = asan
    env["ASAN_OPTIONS"] = "detect_leaks=0:abort_on_error=1:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "print_stacktrace=1:halt_on_error=1"
    env.pop("PYTEST_XDIST_WORKER", None)
    res = subprocess.run([sys.executable, "-c", runner], cwd=ROOT, env=env, stdout=subprocess.PIPE,
                         stderr=subprocess.STDOUT, text=True, timeout=540)
    tail = "\n".join(res.stdout.splitlines()[-40:])
    assert res.returncode == 0, tail
    assert "passed" in tail and "ERROR: AddressSanitizer" not in res.stdout and "runtime error" not in res.stdout, tail
