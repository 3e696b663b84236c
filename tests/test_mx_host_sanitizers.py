"""Argument checks and workspace sizing of routing by a rule and of the microscaled products under
AddressSanitizer and UndefinedBehaviorSanitizer, without a GPU: the ABI file with its host code
instrumented, linked with stand-ins for the launchers and driven from C."""
from __future__ import annotations

import os

import pytest

from test_host_sanitizers import CLANG, CLANGXX, CSRC, ENV, HIPCC, ROOT, _run


def test_mx_abi_under_asan_ubsan(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("the ROCm compilers are not available")
    objs = []
    for src in (os.path.join(CSRC, "qmoe_mx.hip"), os.path.join(ROOT, "tests", "c", "mx_stubs.hip")):
        obj = tmp_path / (os.path.basename(src) + ".o")
        _run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all",
              "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", str(obj)])
        objs.append(str(obj))
    drv = tmp_path / "mx_driver.o"
    _run([CLANG, "-std=c99", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
          "-I", os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", "c", "mx_driver.c"),
          "-o", str(drv)])
    exe = tmp_path / "mx_driver"
    _run([CLANGXX, "-fsanitize=address,undefined", str(drv), *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", str(exe)])
    # the HIP runtime's own start-up allocations are not this library's: leak checks off
    res = _run([str(exe)], env=dict(ENV, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"), timeout=300)
    assert "mx driver: 0 mismatches" in res.stdout
    assert "runtime error" not in res.stderr and "AddressSanitizer" not in res.stderr
