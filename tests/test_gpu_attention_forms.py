"""Attention forms that only large or uneven calls reach: prompt chunks of 8 waves a workgroup in
every type, with pages outside the cache and non-finite values in them; batches of more than 64
prompts; decode splits of fp16 and 8-bit caches; batches that fill the card, whose long
sequences are cut evenly."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

import attn_ref as R
from test_gpu_attention import BF, E4, HF, Case, _plant

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]


def _place(c, row):
    """Sequence of a row and the keys that its sequence has up to it."""
    s = max(i for i in range(len(c.lens)) if c.starts[i] <= row < c.starts[i + 1])
    return s, max(0, c.lens[s]) - (c.starts[s + 1] - row) + 1


def _check_rows(c, got, rows, what, window=0, sinks=0):
    """Some rows of a prefill call against 64 bits, each as a sequence of its own."""
    at = [_place(c, r) for r in rows]
    ref, bound = R.attend(c.q[rows], (c.cache.k, c.cache.v), c.ks, c.vs,
                          torch.stack([c.table[s].cpu() for s, _ in at]), [n for _, n in at],
                          list(range(len(rows) + 1)), 1 / math.sqrt(c.q.shape[-1]), window, sinks,
                          False)
    R.assert_close(got[rows], ref, bound, what)


def _edges(c, count=10, seed=0):
    """First and last rows of every sequence with any, and some between."""
    g = torch.Generator().manual_seed(seed)
    n = c.starts[-1]
    rows = set(torch.randint(0, n, (count,), generator=g).tolist())
    for a, b in zip(c.starts, c.starts[1:]):
        if b > a:
            rows |= {a, b - 1, min(b - 1, a + 63), min(b - 1, a + 64)}
    return sorted(rows)


def _eight_waves(c):
    n, hq, _ = c.q.shape
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert n * hq >= 256 * cus


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D,hq,hkv,page", [(64, 40, 8, 16), (128, 48, 4, 32), (128, 64, 16, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 70), (33, 0)])
def test_large_chunks(D, hq, hkv, page, dtype, cdtype, window, sinks):
    c = Case([1500, 0, 421], [1500, 7, 1001], hq, hkv, D, dtype, cdtype, page, seed=D + page)
    _eight_waves(c)
    _check_rows(c, c.prefill(window=window, sinks=sinks), _edges(c), "chunk", window, sinks)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 16)])
def test_large_chunks_with_pages_outside_the_cache(D, page, dtype, cdtype):
    c = Case([1400, 700], [1400, 1100], 32, 4, D, dtype, cdtype, page, seed=page)
    _eight_waves(c)
    pages = c.cache.k.shape[0]
    for i in (1, 2, 5, 128 // page + 4, 400 // page, 1056 // page):
        c.table[0, i] = -1 if i % 2 else pages
    c.table[1, 0] = 2 ** 31 - 1
    c.table[1, 640 // page: 704 // page + 1] = -2 ** 31
    _check_rows(c, c.prefill(), _edges(c), "pages")
    _check_rows(c, c.prefill(window=200, sinks=5), _edges(c, seed=1), "pages, window", 200, 5)


def _expected(c, hits, window, sinks):
    """Which outputs are not finite when the values at `hits`, (sequence, key, kv head, column),
    are not."""
    n, hq, D = c.q.shape
    group = hq // c.cache.k.shape[1]
    out = torch.zeros((n, hq, D), dtype=torch.bool)
    for seq, key, head, col in hits:
        a, b = c.starts[seq], c.starts[seq + 1]
        pos = c.lens[seq] - (b - a) + torch.arange(b - a)
        sees = (key <= pos) & ((window == 0) | (key > pos - window) | (key < sinks))
        out[a:b, head * group: (head + 1) * group, col] |= sees[:, None]
    return out


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_large_chunks_with_non_finite_values(D, dtype, cdtype):
    lens = [1400, 900]
    c = Case([1400, 700], lens, 32, 4, D, dtype, cdtype, 32, seed=9, fill=float("nan"))
    _eight_waves(c)
    # tiles next to each other and two apart, so that every buffer has some
    hits = [(0, key, key % 4, (5 * key) % D) for key in (3, 70, 133, 257, 258, 700, 1023, 1399)] + \
           [(1, key, key % 4, (3 * key) % D) for key in (0, 199, 200, 201, 330, 899)]
    kinds = [float("nan")] if cdtype == E4 else [float("inf"), float("nan"), -float("inf")]
    for i, hit in enumerate(hits):
        _plant(c, *hit, kinds[i % len(kinds)])
    for window, sinks in ((0, 0), (150, 4)):
        got = c.prefill(window=window, sinks=sinks)
        assert torch.equal(~torch.isfinite(got).cpu(), _expected(c, hits, window, sinks))
        _check_rows(c, got, _edges(c, 16), f"window {window}", window, sinks)


@pytest.mark.parametrize("seqs", [64, 65, 70, 200])
@pytest.mark.parametrize("D,cdtype,long", [(64, BF, 0), (128, E4, 0), (128, BF, 3000), (256, HF, 0)])
def test_many_prompts(seqs, D, cdtype, long):
    # empty prompts among them, at the end too; long contexts split their keys (few tokens)
    dtype = HF if cdtype == HF else BF
    if long:
        qlens = [(i % 3 == 0) * (1 + i % 2) for i in range(seqs)]
        lens = [m + (long * (i + 1)) // seqs for i, m in enumerate(qlens)]
    else:
        qlens = [(i * 7) % 23 * (i % 5 != 3) for i in range(seqs)]
        lens = [m + (i * 13) % 90 for i, m in enumerate(qlens)]
    qlens[-1] = 0
    hq, hkv = (1, 1) if long else (6, 2)
    c = Case(qlens, lens, hq, hkv, D, dtype, cdtype, 16, seed=seqs)
    room = att.prefill_workspace_bytes(c.cache, hq, seqs, sum(qlens), c.table.shape[1])
    assert (room > 0) == (long > 0)
    c.check(c.prefill(), False, "prompts")
    c.check(c.prefill(window=40, sinks=3), False, "prompts, window", window=40, sinks=3)


def test_many_large_prompts():
    # more than 64 prompts and 8 waves a workgroup
    qlens = [(i * 11) % 37 for i in range(90)]
    c = Case(qlens, [m + (i * 29) % 300 for i, m in enumerate(qlens)], 48, 4, 64, BF, BF, 32, seed=5)
    _eight_waves(c)
    c.check(c.prefill(), False, "prompts")


def test_rows_behind_many_prompts_stay():
    qlens = [(i * 7) % 23 for i in range(80)]
    c = Case(qlens, [m + 5 for m in qlens], 4, 2, 64, BF, BF, 16, seed=1)
    out = torch.full_like(c.q, 7.0)
    at = c.starts[70]
    att.attn_prefill(c.cache, c.q, c.int32(c.starts[:71]), c.table[:70], c.int32(c.lens[:70]), out=out)
    assert (out[at:] == 7.0).all() and c.starts[-1] > at
    ref, bound = c.ref(False)
    R.assert_close(out[:at], ref[:at], bound[:at], "rows in front")


@pytest.mark.parametrize("dtype,cdtype", TYPES)
@pytest.mark.parametrize("D,hq,hkv,T", [(64, 8, 1, 2), (128, 4, 2, 1), (128, 16, 1, 4), (256, 8, 2, 2)])
def test_decode_splits_of_all_types(D, hq, hkv, T, dtype, cdtype):
    c = Case([T] * 3, [9011, 40, 1500], hq, hkv, D, dtype, cdtype, 32, seed=3)
    assert att.decode_workspace_bytes(c.cache, hq, 3, T, c.table.shape[1]) > 0
    got = c.decode()
    c.check(got, True, "splits")
    assert torch.equal(c.decode(), got)
    c.check(c.decode(window=2500, sinks=100), True, "splits, window", window=2500, sinks=100)


@pytest.mark.parametrize("dtype,cdtype", TYPES)
def test_even_cuts_of_a_full_batch(dtype, cdtype):
    # the batch fills the card without splits: its long sequences are cut at 4096 keys
    b, hkv = 96, 8
    lens = [(i * 53) % 301 for i in range(b)]
    lens[7], lens[50], lens[95] = 4097, 13000, 8192
    c = Case([1] * b, lens, 16, hkv, 64, dtype, cdtype, 64, seed=12)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert b * hkv > 2 * cus
    splits = att.decode_workspace_bytes(c.cache, 16, b, 1, c.table.shape[1]) // (b * 16 * (64 + 2) * 4)
    assert splits == 4
    c.check(c.decode(), True, "even cuts")
    c.check(c.decode(window=6000, sinks=9), True, "even cuts, window", window=6000, sinks=9)
