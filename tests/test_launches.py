"""What the library hands to the HIP runtime (CPU only, no GPU needed):
tests/c_abi/launch_check.cpp links the built libkda.so with its own functions
in place of the runtime's and looks at every launch."""
import os
import subprocess

import pytest

import gated_delta_rule_25_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CABI = os.path.join(ROOT, "tests", "c_abi")
CLANGXX = "/opt/rocm/llvm/bin/clang++"


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(CLANGXX):
        pytest.skip("ROCm toolchain missing")
    if not os.path.exists(kda._LIB_PATH):
        from gated_delta_rule_25_amd import build
        build.build()
    exe = str(tmp_path_factory.mktemp("launch_check") / "launch_check")
    cmd = [CLANGXX, "-O1", "-g", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "gated_delta_rule_25_amd", "csrc"),
           os.path.join(CABI, "launch_check.cpp"), "-rdynamic", kda._LIB_PATH,
           "-Wl,-rpath," + os.path.dirname(kda._LIB_PATH), "-Wl,-rpath,/opt/rocm/lib", "-Wl,--allow-shlib-undefined",
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


def check(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "launches checked" in r.stdout, r.stdout + r.stderr[-4000:]


def test_calls_without_tokens(program):
    """Such calls take NULL for the tensors of tokens; no kernel may be given
    a constant decay to read at NULL."""
    check(program, "no_tokens")


@pytest.mark.parametrize("what", ["most_stretches", "sizes"])
def test_launches_have_fewer_threads_than_the_runtime_takes(program, what):
    """Fewer than 2^32 a launch, at the sizes the header gives as the largest
    and below them."""
    check(program, what)
