"""Outputs of the dense microscaled product may be columns of the buffer that holds its rows, and
are refused where they share a byte with them. Fake device addresses, never dereferenced: a call
that is not refused fails at its launch (there is no GPU here), which is another status."""
from __future__ import annotations

import ctypes
import random

import pytest
import torch

from quantized_routed_expert_router_amd import mx

INVALID, HIP = 1, 4
BASE = 0x7f0000000000
SIZE = {0: 2, 1: 2, 3: 4}  # bf16, fp16, fp32


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("calls that are not refused would launch on the GPU")


def _call(x, dtype, stride, n, out, out_dtype, out_stride, K=64, N=24):
    w = mx._MxMatrix(BASE + (1 << 40), BASE + (2 << 40), N, K)
    return mx.lib.moe_mx_linear(x, dtype, stride, n, ctypes.byref(w), out, out_dtype, out_stride,
                                BASE + (3 << 40), 1 << 30, None)


@pytest.mark.parametrize("n", [1, 2, 16, 40])
def test_beside_each_other(n):
    # bf16 rows of 64 at columns 32.., 24 fp32 outputs (the width of 48) beside them, 144 columns a row
    x, step = BASE + 64, 144
    # (column 128 ends where the next row begins, column 130 inside it)
    next_row = HIP if n == 1 else INVALID
    for col, want in ((96, HIP), (94, INVALID), (32, INVALID), (-16, HIP), (-14, INVALID), (128, HIP), (130, next_row)):
        assert _call(x, 0, step, n, BASE + 2 * col, 3, step // 2) == want, col
    # another distance between the rows: refused where the ranges meet
    assert _call(x, 0, step, n, BASE + 2 * 96, 3, step // 2 + 1) == (HIP if n == 1 else INVALID)
    assert _call(x, 0, step, n, BASE + 2 * step * n, 3, step // 2 + 1) == HIP


def test_as_bytes_say():
    rng = random.Random(3)
    seen = {HIP: 0, INVALID: 0}
    for _ in range(3000):
        dtype, out_dtype = rng.choice((0, 1, 3)), rng.choice((0, 1, 3))
        K, N, n = 32 * rng.randint(1, 3), rng.randint(1, 40), rng.randint(1, 5)
        step = 16 * rng.randint(1, 40)
        stride, out_stride = step // SIZE[dtype], step // SIZE[out_dtype]
        x, out = BASE + 16 * rng.randint(0, 60), BASE + 4 * rng.randint(0, 240)
        if n > 1 and out_stride < N:
            continue
        xb, ob = K * SIZE[dtype], N * SIZE[out_dtype]
        reads = {b for i in range(n) for b in range(x + i * step, x + i * step + xb)}
        meet = any(b in reads for i in range(n) for b in range(out + i * step, out + i * step + ob))
        got = _call(x, dtype, stride, n, out, out_dtype, out_stride, K, N)
        if meet:
            assert got == INVALID
        elif stride >= K:  # rows that overlap each other are taken by their whole range
            assert got == HIP
        seen[got] += 1
    assert min(seen.values()) > 300
