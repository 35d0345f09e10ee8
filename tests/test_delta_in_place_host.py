"""In-place continuation of the gated delta rule, on the CPU:
tests/c_abi/delta_in_place_check.cpp looks at what the library's launches are
given when the final state takes the initial one's place."""
import os
import subprocess

import pytest

import gated_delta_rule_25_amd as kda
from test_host_sanitize import CABI, CLANGXX, ROOT


def test_no_launch_reads_a_state_that_another_workgroup_of_it_writes(tmp_path):
    if not os.path.exists(CLANGXX):
        pytest.skip("ROCm toolchain missing")
    if not os.path.exists(kda._LIB_PATH):
        from gated_delta_rule_25_amd import build
        build.build()
    exe = str(tmp_path / "delta_in_place_check")
    cmd = [CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "gated_delta_rule_25_amd", "csrc"),
           os.path.join(CABI, "delta_in_place_check.cpp"), "-rdynamic", kda._LIB_PATH,
           "-Wl,-rpath," + os.path.dirname(kda._LIB_PATH), "-Wl,-rpath,/opt/rocm/lib", "-Wl,--allow-shlib-undefined",
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "in-place launches checked" in r.stdout, r.stdout + r.stderr[-4000:]
