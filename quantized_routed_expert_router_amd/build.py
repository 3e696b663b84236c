"""Compile the shared libraries of this package in-tree, the gfx950 ones with hipcc.

Produced next to this file:

* ``libqmoe.so``       - the MoE layer library (C ABI declared in ``include/qmoe.h``);
* ``libqmoe_synth.so`` - the seeded input generator (host and device fill routines);
* ``_fastcall.so``     - the short path of the attention half's Python calls (host code).

Run ``python -m quantized_routed_expert_router_amd.build`` or call :func:`build`.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
JOBS = 8  # compilers at once

# Packed-fp32 VALU forms are disabled for all device code; -ffp-contract=off keeps every
# floating-point multiply and add separately rounded unless a kernel calls fma itself.
COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]

LIBS = {
    "libqmoe.so": ["qmoe.hip", "qmoe_route.hip", "qmoe_decode.hip", "qmoe_prefill.hip",
                   "qmoe_attn.hip", "qmoe_rows.hip", "qmoe_attn_decode.hip",
                   "qmoe_attn_prefill.hip"],
    "libqmoe_synth.so": ["synth.hip"],
}


FASTCALL = "_fastcall.so"


def _fastcall_command(source: str, out: str) -> list[str]:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    includes = [*include_paths(), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-sign-compare",
            f"-D_GLIBCXX_USE_CXX11_ABI={abi}", f"-I{os.path.join(REPO_DIR, 'include')}",
            *(arg for d in includes for arg in ("-isystem", d)), source, "-o", out,
            *(f"-L{d}" for d in library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10",
            f"-L{PKG_DIR}", "-lqmoe", "-Wl,-rpath,$ORIGIN"]


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature name and says so; drop that line
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln]
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {what}:\n" + "\n".join(msgs))
    if msgs and verbose:
        print("\n".join(msgs), flush=True)


def build(verbose: bool = False) -> None:
    """Every source to an object of its own (the sources side by side: they share no device
    code), then one link per library."""
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(JOBS) as pool:
        jobs, objects = [], {}
        for name, sources in LIBS.items():
            objects[name] = [os.path.join(tmp, src + ".o") for src in sources]
            for src, obj in zip(sources, objects[name]):
                cmd = [HIPCC, *COMMON_FLAGS, f"-I{os.path.join(REPO_DIR, 'include')}",
                       f"-I{CSRC}", "-c", os.path.join(CSRC, src), "-o", obj]
                jobs.append(pool.submit(_run, cmd, src, verbose))
        for job in jobs:
            job.result()
        for name, objs in objects.items():
            out = os.path.join(PKG_DIR, name)
            _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", *objs, "-o", out + ".tmp"],
                 name, verbose)
            os.replace(out + ".tmp", out)
    # links against libqmoe.so
    out = os.path.join(PKG_DIR, FASTCALL)
    _run(_fastcall_command(os.path.join(CSRC, "fastcall.cpp"), out + ".tmp"), FASTCALL, verbose)
    os.replace(out + ".tmp", out)


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
