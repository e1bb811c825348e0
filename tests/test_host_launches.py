"""The host code of the 8-bit linear layers and the layer norm under sanitizers, on
the CPU: size queries, kernel choice and launch grids over the documented sizes
(tests/host_launch_check.cpp defines the HIP functions that it calls)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SOURCES = ("api_fp8", "fp8", "gemm_fp8", "api_norm", "norm")


def _run(cmd, **kw):
    p = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert p.returncode == 0, f"{' '.join(cmd)}\n{p.stdout[-4000:]}\n{p.stderr[-4000:]}"
    return p


def test_sizes_and_grids_under_asan_and_ubsan(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    clang = os.path.join(ROCM, "llvm", "bin", "clang++")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not available")
    inc = os.path.join(ROOT, "include")
    objs = []
    for src in SOURCES:  # host pass only: no device code is compiled or run
        objs.append(str(tmp_path / f"{src}.o"))
        _run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-std=c++17", "-fno-pie",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all", "-I", inc,
              "-c", os.path.join(ROOT, "bit_block_float_amd", "csrc", f"{src}.hip"), "-o", objs[-1]])
    driver, exe = str(tmp_path / "driver.o"), str(tmp_path / "host_launch_check")
    _run([clang, "-std=c++17", "-O1", "-g", "-fno-pie", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
          "-D__HIP_PLATFORM_AMD__", "-I", inc, "-I", os.path.join(ROCM, "include"),
          "-c", os.path.join(ROOT, "tests", "host_launch_check.cpp"), "-o", driver])
    # the device code's images are the only symbols left undefined
    _run([clang, "-no-pie", "-fsanitize=address,undefined", driver, *objs, "-Wl,--unresolved-symbols=ignore-all",
          "-o", exe])
    env = dict(os.environ, UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    assert "host-launch-check OK" in _run([exe], env=env, timeout=300).stdout
