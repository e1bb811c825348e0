"""Which kernel a 4-bit product runs, on the CPU: every size of tests/mx4_cases.py
reaches the kernel that it is listed under (tests/mxfp4_choice_check.cpp defines the HIP
functions that the host code calls), and the list has every kernel in every one of its modes."""
import os
import re
import subprocess

import pytest
import torch

import mx4_cases
import mx4_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
SOURCES = ("api_mxfp4", "mxfp4", "gemm_mxfp4")


def _run(cmd, **kw):
    p = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert p.returncode == 0, f"{' '.join(cmd)}\n{p.stdout[-4000:]}\n{p.stderr[-4000:]}"
    return p


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """A function: the kernels of the products, by name, that the calls given as lines launch."""
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    clang = os.path.join(ROCM, "llvm", "bin", "clang++")
    if not (os.path.exists(hipcc) and os.path.exists(clang)):
        pytest.skip("ROCm compilers not available")
    tmp, inc, objs = tmp_path_factory.mktemp("choices"), os.path.join(ROOT, "include"), []
    for src in SOURCES:  # host pass only: no device code is compiled or run
        objs.append(str(tmp / f"{src}.o"))
        _run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17", "-fno-pie", "-I", inc,
              "-c", os.path.join(ROOT, "bit_block_float_amd", "csrc", f"{src}.hip"), "-o", objs[-1]])
    driver, exe = str(tmp / "driver.o"), str(tmp / "choices")
    _run([clang, "-std=c++17", "-O1", "-fno-pie", "-D__HIP_PLATFORM_AMD__", "-I", inc, "-I", os.path.join(ROCM, "include"),
          "-c", os.path.join(ROOT, "tests", "mxfp4_choice_check.cpp"), "-o", driver])
    # the device code's images are the only symbols left undefined
    _run([clang, "-no-pie", driver, *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", exe])

    def run(lines):
        out = _run([exe], input="\n".join(lines) + "\n").stdout.splitlines()
        assert len(out) == len(lines)
        for line in out:
            assert line.endswith("status 0"), line
        return [re.findall(r"_ZN4hif4\d+(mx4_\S+)", line) for line in out]

    return run


def _check(launches, cases, lines):
    for case, line, got in zip(cases, lines, launches(lines)):
        assert len(got) == len(case[0]) and all(g.startswith(k) for g, k in zip(got, case[0])), (line, case[0], got)


def test_linear(launches):
    _check(launches, mx4_cases.LINEAR, [f"linear {m} {n} {k}" for _, m, n, k in mx4_cases.LINEAR])


def test_grouped(launches):
    _check(launches, mx4_cases.GROUPED,
           [f"grouped {len(o) - 1} {m} {n} {k}" for _, m, o, n, k in mx4_cases.GROUPED])


def test_backward(launches):
    _check(launches, mx4_cases.BACKWARD, [f"backward {m} {n} {k} {w}" for _, m, n, k, w in mx4_cases.BACKWARD])


def test_grouped_backward(launches):
    _check(launches, mx4_cases.GROUPED_BACKWARD,
           [f"grouped_backward {len(o) - 1} {m} {n} {k} {w}" for _, m, o, n, k, w in mx4_cases.GROUPED_BACKWARD])


def test_every_kernel_is_listed():
    c = mx4_cases
    reached = lambda cases: {k for case in cases for k in case[0]}  # noqa: E731
    assert reached(c.LINEAR) == {c.SKINNY16, c.SKINNY32, c.T64, c.T128, c.T256, c.SPLIT}
    assert reached(c.GROUPED) == {c.SKINNY32, c.T64, c.T128, c.T256}
    assert reached(c.BACKWARD) == {c.SKINNY16, c.SKINNY32, c.T64, c.T128, c.T256, c.SPLIT}
    only = [case for case in c.GROUPED_BACKWARD if case[-1] == 2]  # K by groups
    assert reached(only) == {c.T64, c.T128, c.T256}


def test_rounded_is_what_codes_and_scales_stand_for():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((300, 500), generator=g) * torch.exp(3 * torch.randn((1, 500), generator=g))
    x[0], x[1] = 0.0, 2.0 ** -130
    x[2:10, ::32] = 6.0
    x[2:10, 1:33] = torch.arange(-32, 0) / 8  # ties
    for t in (x, x.T, x.to(torch.bfloat16)):
        assert torch.equal(mx4_cases.rounded(t), mx4_ref.values(*mx4_ref.quantize(t)))
