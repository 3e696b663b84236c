"""The tile list's split over the XCDs, by the library's own functions compiled for the host."""
from __future__ import annotations

import os

import pytest

from test_host_sanitizers import CSRC, HIPCC, ROOT, _run


def test_split_of_the_tile_list(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("the ROCm compiler is not available")
    exe = tmp_path / "mx_split"
    _run([HIPCC, "--offload-host-only", "-std=c++17", "-O2", "-Wall", "-Wno-unused-function",
          "-I", os.path.join(ROOT, "include"), "-I", CSRC,
          os.path.join(ROOT, "tests", "c", "mx_split_driver.hip"), "-o", str(exe)])
    assert "mx split: 0 failures" in _run([str(exe)], timeout=120).stdout
