"""Decode attention with page tables far wider than the sequences are long, and batches of very
different lengths: the split of the keys follows the lengths, not the table."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

import attn_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [0, 64, 2048])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 9)])
def test_wide_tables_and_uneven_lengths(width, window, sinks):
    g = torch.Generator().manual_seed(3)
    lens = [5000, 1, 0, 257, 4097, 33, 2048, 900]
    hq, hkv, D, page, T = 4, 2, 64, 32, 2
    need = [-(-n // page) for n in lens]
    pages = sum(need)
    k = torch.randn((pages, hkv, page, D), generator=g).bfloat16().cuda()
    v = torch.randn((pages, hkv, page // 8, D, 8), generator=g).bfloat16().cuda()
    table = torch.full((len(lens), max(need) + width), 1 << 30, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at: at + m]
        at += m
    q = torch.randn((len(lens) * T, hq, D), generator=g).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    got = att.attn_decode(att.KVCache(k, v), q, table.cuda(), n, window=window, sinks=sinks)
    ref, bound = R.attend(q, (k, v), None, None, table, lens, [T * i for i in range(len(lens) + 1)],
                          1 / math.sqrt(D), window, sinks, True)
    R.assert_close(got, ref, bound, f"width {width}")
