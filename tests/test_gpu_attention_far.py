"""Positions behind 2^30: windows and first keys of 2^30 and more hide exactly what they say.
A page table may name a page more than once, so a context of that length fits one small
cache."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

pytestmark = pytest.mark.gpu

PAGE, D = 256, 64
L = (1 << 30) + (1 << 20)


def _cache():
    """Page 0: keys of score 0 and value 0; page 1 the same but for its row 0, of score 24 and
    value 1."""
    cache = att.KVCache.empty(2, 1, PAGE, D)
    cache.k.zero_()
    cache.v.zero_()
    cache.k[1, 0, 0, 0] = 1
    cache.v[1, 0, 0, :, 0] = 1
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 24
    return cache, q


# window, sinks, the key with the value, whether the last token sees it, and how many others
CASES = [
    (2 ** 31 - 1, 0, 0, True, L),                   # a window longer than the context hides nothing
    (L, 0, 0, True, L),                             # exactly as long
    (L - 256, 0, 0, False, L - 256),                # the first page lies behind it
    (1 << 30, 0, 0, False, 1 << 30),
    ((1 << 30) + 512, 0, (1 << 20) - 512, True, (1 << 30) + 512),  # its oldest key
    (16, 2 ** 31 - 1, (1 << 30) + 1024, True, L),   # every key is a first key
]


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("window,sinks,key,seen,keys", CASES)
def test_window_at_far_positions(kind, window, sinks, key, seen, keys):
    cache, q = _cache()
    table = torch.zeros((1, L // PAGE), dtype=torch.int32, device="cuda")
    assert key % PAGE == 0
    table[0, key // PAGE] = 1
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    if kind == "decode":
        out = att.attn_decode(cache, q, table, lens, scale=1.0, window=window, sinks=sinks)
    else:
        starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        out = att.attn_prefill(cache, q, starts, table, lens, scale=1.0, window=window, sinks=sinks)
    want = math.exp(24) / (math.exp(24) + keys - 1) if seen else 0.0
    # the sums: 2^-11 at most (fp32 sums of equal terms over 2^18 keys a lane, exact up to 2^24,
    # and a few roundings); the output's rounding: 2^-8
    assert (out.double() - want).abs().max().item() <= want * (2.0 ** -8 + 2.0 ** -11)
