"""The attention half without a GPU: the C ABI's argument checks and workspace sizing (driven
from C, once against the built library and once under AddressSanitizer and
UndefinedBehaviorSanitizer on the host code), the binding's struct layouts, and the binding's
own checks. No kernel is launched."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att
from quantized_routed_expert_router_amd import qmoe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_routed_expert_router_amd", "csrc")
DRIVER = os.path.join(ROOT, "tests", "c", "attn_driver.c")
HIPCC, CLANG, CLANGXX = ("/opt/rocm/bin/hipcc", "/opt/rocm/llvm/bin/clang",
                         "/opt/rocm/llvm/bin/clang++")


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert res.returncode == 0, f"{' '.join(cmd)}\n{res.stdout}\n{res.stderr}"
    return res.stdout


@pytest.fixture(scope="module")
def driver_output(tmp_path_factory):
    if shutil.which("gcc") is None:
        pytest.skip("gcc is not available")
    exe = str(tmp_path_factory.mktemp("attn") / "driver")
    libdir = os.path.dirname(qmoe.LIB_PATH)
    _run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
          os.path.join(ROOT, "include"), DRIVER, "-L", libdir, "-lqmoe", f"-Wl,-rpath,{libdir}",
          "-o", exe])
    return _run([exe], timeout=120)


def test_rejected_calls(driver_output):
    assert "attention driver: 0 mismatches" in driver_output


@pytest.mark.parametrize("name,struct", [
    ("moe_heads", att._Heads), ("moe_kv_cache", att._KVCache), ("moe_norm_rope", att._NormRope),
    ("moe_pages", att._Pages), ("moe_attn", att._Attn)])
def test_struct_layouts(driver_output, name, struct):
    assert f"sizeof {name} {ctypes.sizeof(struct)}\n" in driver_output


def test_host_side_under_asan_ubsan(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("the ROCm compilers are not available")
    objs = []
    for src in (os.path.join(CSRC, "qmoe.hip"), os.path.join(CSRC, "qmoe_attn.hip"),
                os.path.join(ROOT, "tests", "c", "launch_stubs.hip"),
                os.path.join(ROOT, "tests", "c", "attn_stubs.hip")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"),
              "-I", CSRC, "-c", src, "-o", obj])
        objs.append(obj)
    drv = str(tmp_path / "driver.o")
    _run([CLANG, "-std=c99", "-O1", "-g", "-fsanitize=address,undefined",
          "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-c", DRIVER, "-o", drv])
    exe = str(tmp_path / "driver")
    _run([CLANGXX, "-fsanitize=address,undefined", drv, *objs, "-L/opt/rocm/lib", "-lamdhip64",
          "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    assert "attention driver: 0 mismatches" in _run([exe], env=env, timeout=300)


# ------------------------------------------------------------------ the binding

BF = torch.bfloat16


def _cache(pages=4, heads=2, page=16, D=64, dtype=BF):
    return att.KVCache.empty(pages, heads, page, D, dtype, device="cpu")


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _q(n=3, heads=4, D=64, dtype=BF):
    return torch.zeros(n, heads, D, dtype=dtype)


def test_host_tensors_are_rejected():
    for call in (lambda: att.qk_norm_rope(_q(), _q(heads=2), None, att.NormRope()),
                 lambda: att.kv_append(_cache(), _q(heads=2), _q(heads=2), _i32(3)),
                 lambda: att.attn_decode(_cache(), _q(), _i32(3, 4), _i32(3)),
                 lambda: att.attn_prefill(_cache(), _q(), _i32(2), _i32(1, 4), _i32(1))):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call()


def test_norm_rope_checks():
    rope = lambda q=_q(), k=_q(heads=2), pos=_i32(3), p=att.NormRope(), **kw: (  # noqa: E731
        att.qk_norm_rope(q, k, pos, p, **kw))
    with pytest.raises(ValueError, match="at least one"):
        rope(q=None, k=None)
    with pytest.raises(ValueError, match="q: dtype"):
        rope(q=_q(dtype=torch.float32))
    with pytest.raises(ValueError, match="k: dtype"):
        rope(k=_q(heads=2, dtype=torch.float16))
    with pytest.raises(ValueError, match="k: shape"):
        rope(k=_q(n=2, heads=2))
    with pytest.raises(ValueError, match="q: expected"):
        rope(q=torch.zeros(3, 256, dtype=BF))
    with pytest.raises(ValueError, match="q: the last axis"):
        rope(q=torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2), k=None)
    with pytest.raises(ValueError, match="positions: dtype"):
        rope(pos=_i32(3).long())
    with pytest.raises(ValueError, match="positions: shape"):
        rope(pos=_i32(4))
    with pytest.raises(ValueError, match="q_norm: shape"):
        rope(p=att.NormRope(q_norm=torch.ones(32)))
    with pytest.raises(ValueError, match="inv_freq: dtype"):
        rope(p=att.NormRope(inv_freq=torch.ones(32, dtype=torch.float64)))
    with pytest.raises(ValueError, match="q_out: shape"):
        rope(q_out=_q(heads=3))
    with pytest.raises(ValueError, match="k_out: given without"):
        rope(k=None, k_out=_q(heads=2))


def test_append_checks():
    call = lambda c=_cache(), k=_q(heads=2), v=_q(heads=2), s=_i32(3), **kw: (  # noqa: E731
        att.kv_append(c, k, v, s, **kw))
    with pytest.raises(ValueError, match="v: shape"):
        call(v=_q(heads=3))
    with pytest.raises(ValueError, match="k: shape"):
        call(c=_cache(heads=3))
    with pytest.raises(ValueError, match="slots: shape"):
        call(s=_i32(2))
    with pytest.raises(ValueError, match="slots: dtype"):
        call(s=_i32(3).long())
    with pytest.raises(ValueError, match="q: needs p"):
        call(q=_q())
    with pytest.raises(ValueError, match="q_out: given without q"):
        call(q_out=_q())
    c = _cache()
    with pytest.raises(ValueError, match="cache.v: shape"):
        call(c=att.KVCache(c.k, c.k))
    with pytest.raises(ValueError, match="cache.k: dtype"):
        call(c=att.KVCache(c.k.float(), c.v))
    with pytest.raises(ValueError, match="cache.k_scale: shape"):
        call(c=att.KVCache(c.k, c.v, k_scale=torch.ones(3)))
    with pytest.raises(ValueError, match="page_size"):
        att.KVCache.empty(1, 1, 12, 64, device="cpu")


def test_attention_checks():
    dec = lambda c=_cache(), q=_q(), t=_i32(3, 4), n=_i32(3), **kw: (  # noqa: E731
        att.attn_decode(c, q, t, n, **kw))
    with pytest.raises(ValueError, match="q: head_dim"):
        dec(q=_q(D=128))
    with pytest.raises(ValueError, match="multiple of 3 sequences"):
        dec(q=_q(n=4))
    with pytest.raises(ValueError, match="page_table: dtype"):
        dec(t=_i32(3, 4).long())
    with pytest.raises(ValueError, match="page_table: expected"):
        dec(t=_i32(12))
    with pytest.raises(ValueError, match="page_table: the last axis"):
        dec(t=_i32(4, 3).t())
    with pytest.raises(ValueError, match="page_table: rows overlap"):
        dec(t=_i32(1, 4).expand(3, 4))
    with pytest.raises(ValueError, match="kv_lens: shape"):
        dec(n=_i32(2))
    with pytest.raises(ValueError, match="window, sinks"):
        dec(window=-1)
    with pytest.raises(ValueError, match="window, sinks"):
        dec(sinks=1 << 31)
    with pytest.raises(ValueError, match="out: shape"):
        dec(out=_q(n=2))
    with pytest.raises(ValueError, match="ws: dtype"):
        dec(ws=torch.zeros(4))
    with pytest.raises(ValueError, match="q_starts: expected"):
        att.attn_prefill(_cache(), _q(), None, _i32(1, 4), _i32(1))
    with pytest.raises(ValueError, match="q_starts: shape"):
        att.attn_prefill(_cache(), _q(), _i32(3), _i32(1, 4), _i32(1))


def test_workspace_queries():
    c = _cache(pages=4096)
    assert att.decode_workspace_bytes(c, 4, 1, 1, 8) == 0       # a short context: one split
    long = att.decode_workspace_bytes(c, 4, 1, 1, 4096)
    assert long > 0 and long % 256 == 0
    # a window bounds what a call can see, and so its splits
    assert att.decode_workspace_bytes(c, 4, 1, 1, 4096, window=64, sinks=4) == 0
    assert att.prefill_workspace_bytes(c, 4, 1, 20, 4096) > 0
    assert att.prefill_workspace_bytes(c, 64, 1, 8192, 4096) == 0
    assert att.prefill_workspace_bytes(c, 4, 1, 8193, 4096) == 0  # out of range
