"""Precondition checks of two threads at once (CPU): tests/c_abi/check_threads.cpp."""
import os
import subprocess

import pytest

import gated_delta_rule_25_amd as kda
from test_host_sanitize import CABI, CLANGXX, ROOT


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(CLANGXX):
        pytest.skip("ROCm toolchain missing")
    if not os.path.exists(kda._LIB_PATH):
        from gated_delta_rule_25_amd import build
        build.build()
    exe = str(tmp_path_factory.mktemp("check_threads") / "check_threads")
    cmd = [CLANGXX, "-O1", "-g", "-std=c++17", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), os.path.join(CABI, "check_threads.cpp"), "-rdynamic", kda._LIB_PATH,
           "-Wl,-rpath," + os.path.dirname(kda._LIB_PATH), "-Wl,-rpath,/opt/rocm/lib", "-Wl,--allow-shlib-undefined",
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.parametrize("which", [0, 1, 2], ids=["kda", "linear", "delta"])
def test_each_thread_gets_its_own_answer(program, which):
    r = subprocess.run([program, str(which)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
