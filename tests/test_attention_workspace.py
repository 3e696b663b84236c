"""Workspace of decode attention: a page table says how long a sequence may be, not how long it
is, so its width must not make a call's workspace grow without end."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att
from quantized_routed_expert_router_amd.qmoe import lib

import attn_ref as R

LIMIT = (256 << 20) + 512  # and the alignment of its two parts


def _bytes(seqs, tokens, q_heads, kv_heads, D, keys, page=64, window=0):
    cache = att._KVCache(0, 0, 0, 0, 0, 4, page, kv_heads, D)
    a = att._Attn(1.0, window, 0)
    return lib.moe_attn_decode_workspace_bytes(ctypes.byref(cache), q_heads, seqs, tokens,
                                               keys // page, ctypes.byref(a))


@pytest.mark.parametrize("seqs,tokens", [(1, 1), (1, 16), (7, 4), (32, 16), (64, 8), (128, 4), (512, 1)])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (1, 64), (1, 512), (8, 4), (8, 8), (64, 8), (512, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bounded_whatever_the_table(seqs, tokens, kv_heads, group, D):
    for keys in (1 << 10, 1 << 15, 1 << 18, 1 << 20, 1 << 24, 1 << 30):
        for window in (0, 1 << 20):
            assert _bytes(seqs, tokens, kv_heads * group, kv_heads, D, keys, window=window) <= LIMIT


def test_splits_of_usual_calls():
    parts = lambda *a: _bytes(*a) / (a[0] * a[1] * a[2] * (4 * a[4] + 8))  # noqa: E731
    # one long sequence still fills the card, and uneven batches are still cut at 4096 keys
    assert round(parts(1, 4, 16, 2, 256, 1 << 18)) >= 128
    assert round(parts(64, 1, 32, 8, 128, 32768)) == 8
    assert round(parts(64, 1, 32, 8, 128, 1 << 18)) == 64


@pytest.mark.parametrize("kv_heads,group", [(1, 8), (2, 8), (8, 4), (8, 12), (3, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_large_prompt_chunks_take_no_workspace(kv_heads, group, D):
    # chunks of 256 rows a workgroup fill the card and never split their keys
    cache = att._KVCache(0, 0, 0, 0, 0, 4, 64, kv_heads, D)
    a = att._Attn(1.0, 0, 0)
    heads = kv_heads * group
    for n in (-(-65536 // heads), 8192):
        for seqs in (1, 5, 300, 8192):
            if n * heads >= 65536 and n <= 8192:
                assert lib.moe_attn_prefill_workspace_bytes(ctypes.byref(cache), heads, seqs, n,
                                                            1 << 14, ctypes.byref(a)) == 0


@pytest.mark.gpu
def test_long_sequence_in_a_batch_at_the_bound():
    g = torch.Generator().manual_seed(11)
    b, T, hq, hkv, D, page = 128, 4, 16, 2, 64, 256
    lens = [(37 * i) % 700 for i in range(b)]
    lens[5], lens[90] = 30011, 9000
    need = [-(-n // page) for n in lens]
    pages = sum(need)
    k = torch.randn((pages, hkv, page, D), generator=g).bfloat16().cuda()
    v = torch.randn((pages, hkv, page // 8, D, 8), generator=g).bfloat16().cuda()
    table = torch.full((b, (1 << 20) // page), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at: at + m]
        at += m
    cache = att.KVCache(k, v)
    room = att.decode_workspace_bytes(cache, hq, b, T, table.shape[1])
    assert LIMIT // 2 < room <= LIMIT
    q = torch.randn((b * T, hq, D), generator=g).bfloat16().cuda()
    got = att.attn_decode(cache, q, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    ref, bound = R.attend(q, (k, v), None, None, table, lens, [T * i for i in range(b + 1)],
                          1 / math.sqrt(D), 0, 0, True)
    R.assert_close(got, ref, bound, "batch")
