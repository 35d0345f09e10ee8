"""Host code of include/kda_linear.h and include/kda_beam.h under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only, no GPU needed):
kda_linear_api.hip and kda_beam_api.hip, sanitized on their host side, with
tests/c_abi/linear_host_sanitize.cpp in place of the kernels' launches."""
import os
import subprocess

import pytest

from test_host_sanitize import CABI, CLANGXX, HIPCC, INC, ROOT, SAN, _host_san


@pytest.mark.skipif(not all(os.path.exists(x) for x in (HIPCC, CLANGXX)), reason="ROCm toolchain missing")
def test_linear_and_beam_host_code(tmp_path):
    base = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-Xclang", "-target-feature", "-Xclang",
            "-packed-fp32-ops"]
    objs, steps = [], []
    for name in ("kda_linear_api", "kda_beam_api"):
        objs.append(str(tmp_path / (name + ".o")))
        steps.append([HIPCC] + base + _host_san() + INC +
                     ["-c", os.path.join(ROOT, "gated_delta_rule_25_amd", "csrc", name + ".hip"), "-o", objs[-1]])
    exe = str(tmp_path / "linear_host_sanitize")
    objs.append(str(tmp_path / "drv.o"))
    steps.append([CLANGXX, "-O1", "-g", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"] + SAN +
                 INC + ["-c", os.path.join(CABI, "linear_host_sanitize.cpp"), "-o", objs[-1]])
    steps.append([CLANGXX] + SAN + objs + ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    for cmd in steps:
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, "build step failed:\n" + " ".join(cmd) + "\n" + r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert r.returncode == 0 and "linear host sanitizer checks passed" in out, out[-4000:]
