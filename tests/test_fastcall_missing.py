"""Without _fastcall.so (it links against one build of torch): routing and the block-quantized
layer, which never used it, still import; what needs it says so."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "quantized_routed_expert_router_amd"


def _run(body: str) -> str:
    # None in sys.modules is how Python marks a module that cannot be imported
    code = f"import sys\nsys.modules['{PKG}._fastcall'] = None\n{body}"
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    return res.stdout


def test_plain_calls_import_without_it():
    out = _run(f"from {PKG} import qmoe, synth, workloads\nimport torch\n"
               "print(qmoe.status_string(0), qmoe.lib.moe_route_workspace_bytes(8192, 512, 10))\n"
               "try: qmoe.route(torch.zeros(3, 8), 2, out=qmoe.Routing.empty(3, 8, 2, 'cpu'))\n"
               "except ValueError as e: print(e)")
    assert out.splitlines()[0] == f"MOE_OK {40 * 512 * 4}" and "must be a GPU tensor" in out


@pytest.mark.parametrize("module", ["mx", "attention"])
def test_modules_that_need_it_say_so(module):
    out = _run(f"try: from {PKG} import {module}\nexcept ImportError as e: print(e)")
    assert "_fastcall.so is missing or does not load" in out


def test_the_call_that_needs_it_says_so():
    # a stand-in for a tensor on a GPU: the short path is looked for before anything is read
    out = _run(f"from {PKG} import qmoe\nimport torch\n"
               "qmoe._current_device = lambda: 0\n"
               "torch.Tensor.is_cuda = True\n"
               "try: qmoe.route_scored(torch.zeros(3, 8), 2, qmoe.RouteRule())\nexcept ImportError as e: print(e)")
    assert "_fastcall.so is missing or does not load" in out
