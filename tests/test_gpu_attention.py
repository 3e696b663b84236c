"""Decode-window and prefill-chunk attention over the paged cache against the 64-bit
formulas: types, head layouts, page sizes, lengths, windows and first keys, non-finite
values behind masks, pages outside the cache."""
from __future__ import annotations

import math

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

import attn_ref as R

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


class Case:
    """A cache with shuffled pages and the sequences' tables; unused rows hold `fill`."""

    def __init__(self, qlens, lens, hq, hkv, D, dtype, cdtype, page, seed=0, fill=None, extra=2,
                 width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(0, x) // page) for x in lens]
        pages = sum(need) + extra
        ck = torch.randn((pages, hkv, page, D), generator=g)
        cv = torch.randn((pages, hkv, page, D), generator=g) + 0.25
        order = torch.randperm(pages, generator=g)
        width = width or max(1, max(need) + 1)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        used = torch.zeros((pages, page), dtype=torch.bool)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at: at + m]
            key = torch.arange(max(0, lens[i]))
            used[table[i].long()[key // page], key % page] = True
            at += m
        if fill is not None:
            ck.transpose(1, 2)[~used] = fill
            cv.transpose(1, 2)[~used] = fill
        cv = cv.view(pages, hkv, page // 8, 8, D).transpose(3, 4).contiguous()
        self.ks = self.vs = None
        if cdtype == E4:
            self.ks = (0.5 + torch.rand(hkv, generator=g)).cuda()
            self.vs = (0.5 + torch.rand(hkv, generator=g)).cuda()
        self.cache = att.KVCache(ck.to(cdtype).cuda(), cv.to(cdtype).cuda(), self.ks, self.vs)
        self.q = torch.randn((sum(qlens), hq, D), generator=g).to(dtype).cuda()
        self.table = table.cuda()
        self.lens = list(lens)
        self.starts = [sum(qlens[:i]) for i in range(len(qlens) + 1)]

    def ref(self, two_part, window=0, sinks=0, scale=None):
        scale = 1 / math.sqrt(self.q.shape[-1]) if scale is None else scale
        return R.attend(self.q, (self.cache.k, self.cache.v), self.ks, self.vs, self.table.cpu(),
                        self.lens, self.starts, scale, window, sinks, two_part)

    def int32(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def decode(self, **kw):
        return att.attn_decode(self.cache, self.q, self.table, self.int32(self.lens), **kw)

    def prefill(self, **kw):
        return att.attn_prefill(self.cache, self.q, self.int32(self.starts), self.table,
                                self.int32(self.lens), **kw)

    def check(self, got, two_part, what, **kw):
        ref, bound = self.ref(two_part, **kw)
        R.assert_close(got, ref, bound, what)


LENS = [0, 1, 2, 31, 32, 33, 64, 257, 700]


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("D,hq,hkv,T,page", [
    (64, 1, 1, 1, 16), (64, 40, 8, 5, 32), (128, 8, 2, 4, 16), (128, 32, 8, 1, 64),
    (128, 12, 1, 7, 128), (256, 16, 2, 4, 64), (256, 3, 3, 1, 16), (256, 10, 1, 16, 256),
    (64, 16, 1, 8, 16),
])
def test_decode(D, hq, hkv, T, page, dtype, cdtype):
    c = Case([T] * len(LENS), LENS, hq, hkv, D, dtype, cdtype, page, seed=D + T)
    c.check(c.decode(), True, "decode")


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (32, 0), (33, 40), (100, 4), (5000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("D,cdtype,page", [(128, BF, 16), (64, E4, 64)])
def test_decode_window(window, sinks, D, cdtype, page):
    lens = [0, 3, 64, 130, 1500]
    c = Case([4] * 5, lens, 8, 2, D, BF, cdtype, page, seed=window % 97)
    c.check(c.decode(window=window, sinks=sinks), True, "window", window=window, sinks=sinks)


@pytest.mark.parametrize("D,cdtype", [(128, BF), (256, BF), (64, E4)])
def test_decode_splits(D, cdtype):
    # one long and one short sequence: many splits that are joined, beside a single one
    c = Case([2, 2], [20011, 40], 8, 1, D, BF, cdtype, 32, seed=3)
    assert att.decode_workspace_bytes(c.cache, 8, 2, 2, c.table.shape[1]) > 0
    got = c.decode()
    c.check(got, True, "splits")
    for _ in range(3):
        assert torch.equal(c.decode(), got)  # the same bits every time
    win = c.decode(window=9000, sinks=100)
    c.check(win, True, "splits with a window", window=9000, sinks=100)


PREFILL = [
    # qlens, lens, hq, hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([37], [37], 16, 4, 64, 16),
    ([5, 0, 1, 130, 64], [5, 9, 300, 131, 64], 8, 2, 128, 32),
    ([33, 200], [1000, 200], 6, 2, 256, 64),
    ([7, 3, 9], [3, 0, 9], 5, 5, 128, 16),  # fewer keys than tokens
    ([300], [777], 12, 1, 64, 256),
    ([257, 129], [400, 129], 3, 1, 128, 128),
]


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (HF, HF), (BF, E4), (HF, E4)])
@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill(i, dtype, cdtype):
    qlens, lens, hq, hkv, D, page = PREFILL[i]
    c = Case(qlens, lens, hq, hkv, D, dtype, cdtype, page, seed=i)
    c.check(c.prefill(), False, "prefill")


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 2), (64, 0), (65, 70), (300, 4),
                                          (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("D,cdtype,page", [(128, BF, 16), (64, E4, 64), (256, BF, 32)])
def test_prefill_window(window, sinks, D, cdtype, page):
    c = Case([150, 20, 1], [150, 900, 333], 4, 2, D, BF, cdtype, page, seed=window % 89)
    c.check(c.prefill(window=window, sinks=sinks), False, "window", window=window, sinks=sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_splits(D):
    # few rows over a long context: split keys, joined; beside it a chunk with one split
    c = Case([9, 30], [9000, 30], 4, 1, D, BF, BF, 64, seed=D)
    assert att.prefill_workspace_bytes(c.cache, 4, 2, 39, c.table.shape[1]) > 0
    got = c.prefill()
    c.check(got, False, "splits")
    for _ in range(3):
        assert torch.equal(c.prefill(), got)


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_many_rows(D):
    # enough rows for the 8-wave workgroups
    c = Case([1100, 421], [1100, 600], 48, 8, D, BF, BF, 64, seed=D)
    c.check(c.prefill(), False, "many rows")
    c.check(c.prefill(window=200, sinks=3), False, "many rows, window", window=200, sinks=3)


def test_prefill_rows_behind_the_last_sequence_stay():
    c = Case([20, 13, 30], [20, 50, 30], 4, 2, 128, BF, BF, 16, seed=4)
    out = torch.full_like(c.q, 7.0)
    starts = c.int32([0, 20, 33])
    att.attn_prefill(c.cache, c.q, starts, c.table[:2], c.int32(c.lens[:2]), out=out)
    assert (out[33:] == 7.0).all()
    ref, bound = c.ref(False)
    R.assert_close(out[:33], ref[:33], bound[:33], "rows in front")


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,cdtype", [(128, BF), (64, HF), (256, BF), (128, E4)])
def test_rows_behind_the_keys_do_not_matter(D, cdtype, fill):
    dtype = HF if cdtype == HF else BF
    lens = [1, 17, 45, 500]
    c = Case([3] * 4, lens, 4, 2, D, dtype, cdtype, 16, fill=fill)
    c.check(c.decode(), True, "decode")
    c = Case([1, 17, 40, 100], lens, 4, 2, D, dtype, cdtype, 16, fill=fill)
    c.check(c.prefill(), False, "prefill")


def _plant(c, seq, key, head, col, value):
    page = c.cache.k.shape[2]
    pg, r = int(c.table[seq, key // page]), key % page
    c.cache.v[pg, head, r // 8, col, r % 8] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_non_finite_values_reach_only_rows_that_see_them(D, value):
    # key 99 is seen by the last token alone, key 20 by every token (outside the window: none)
    c = Case([4], [100], 4, 2, D, BF, BF, 16)
    _plant(c, 0, 99, 1, 5, value)
    c.check(c.decode(), True, "decode, last key")
    _plant(c, 0, 20, 0, 3, value)
    c.check(c.decode(), True, "decode, seen by all")
    c.check(c.decode(window=40, sinks=2), True, "decode, outside the window", window=40, sinks=2)
    c.check(c.decode(window=78, sinks=2), True, "decode, at the window", window=78, sinks=2)
    c = Case([60], [100], 4, 2, D, BF, BF, 16)
    _plant(c, 0, 70, 1, 5, value)
    _plant(c, 0, 99, 0, D - 1, value)
    c.check(c.prefill(), False, "prefill")
    c.check(c.prefill(window=20, sinks=2), False, "prefill, window", window=20, sinks=2)


def test_non_finite_queries_and_keys():
    # a NaN query row is NaN alone; a key that scores NaN spoils the rows that see it
    c = Case([6], [40], 4, 2, 64, BF, BF, 16)
    c.q[2, 1, 7] = float("nan")
    ref, bound = c.ref(True)
    assert torch.isnan(ref[2, 1]).all() and torch.isfinite(ref[3]).all()
    R.assert_close(c.decode(), ref, bound, "decode")
    ref, bound = c.ref(False)
    R.assert_close(c.prefill(), ref, bound, "prefill")
    c = Case([6], [40], 4, 2, 64, BF, BF, 16)
    page = c.cache.k.shape[2]
    c.cache.k[int(c.table[0, 37 // page]), 0, 37 % page, 3] = float("nan")
    for got in (c.decode(), c.prefill()):
        assert torch.isnan(got[3:, :2]).all()       # heads 0, 1 read kv head 0; tokens 37..39
        assert torch.isfinite(got[:3]).all() and torch.isfinite(got[:, 2:]).all()


@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_cache_count_as_unseen(page):
    lens = [5 * page + 3, 2 * page]
    c = Case([4, 4], lens, 4, 2, 128, BF, BF, page)
    pages = c.cache.k.shape[0]
    c.table[0, 1], c.table[0, 3] = -1, pages
    c.table[1] = 2 ** 31 - 1  # no page at all: zeros
    got = c.decode()
    c.check(got, True, "decode")
    assert (got[4:] == 0).all()
    got = c.prefill()
    c.check(got, False, "prefill")
    assert (got[4:] == 0).all()


def test_pages_outside_the_window_are_not_read():
    # their entries hold anything
    c = Case([4], [1000], 4, 2, 128, BF, BF, 16)
    want = c.decode(window=100, sinks=5)
    want_p = c.prefill(window=100, sinks=5)
    c.table[0, 1: (1000 - 104) // 16] = 2 ** 31 - 1
    assert torch.equal(c.decode(window=100, sinks=5), want)
    assert torch.equal(c.prefill(window=100, sinks=5), want_p)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_scales(scale):
    c = Case([5], [70], 4, 2, 64, BF, BF, 16)
    c.check(c.decode(scale=scale), True, "decode", scale=scale)
    c.check(c.prefill(scale=scale), False, "prefill", scale=scale)


def test_large_scores():
    # one key far above the others, and rows whose maximum moves from tile to tile
    c = Case([4], [600], 4, 2, 128, BF, BF, 16, seed=2)
    c.q *= 8
    c.check(c.decode(), True, "decode")
    c.check(c.prefill(), False, "prefill")


def test_strided_queries_and_tables():
    c = Case([2, 2], [90, 33], 4, 2, 64, BF, BF, 16)
    wide = torch.zeros((4, 3 * 4 * 64), dtype=BF, device="cuda")
    q = wide[:, 4 * 64: 8 * 64].view(4, 4, 64)
    q.copy_(c.q)
    table = torch.full((2, 40), -7, dtype=torch.int32, device="cuda")
    table[:, 3: 3 + c.table.shape[1]] = c.table
    view = table[:, 3: 3 + c.table.shape[1]]
    got = att.attn_decode(c.cache, q, view, c.int32(c.lens))
    assert torch.equal(got, c.decode())
    got = att.attn_prefill(c.cache, q, c.int32(c.starts), view, c.int32(c.lens))
    assert torch.equal(got, c.prefill())
    heads_first = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(att.attn_decode(c.cache, heads_first, c.table, c.int32(c.lens)), c.decode())


def test_offsets_past_32_bits():
    # the sequence's pages lie behind 2^31 elements of the cache
    pages, hkv, page, D = (1 << 31) // (8 * 64 * 128) + 64, 8, 64, 128
    assert pages * hkv * page * D > 1 << 31
    cache = att.KVCache.empty(pages, hkv, page, D, BF)
    n = 70
    k, v, q = (_rand((n, h, D), BF, s) for h, s in ((hkv, 1), (hkv, 2), (16, 3)))
    ids = torch.tensor([pages - 1, pages - 5], dtype=torch.int32)
    slots = torch.cat([ids[0] * page + torch.arange(64), ids[1] * page + torch.arange(6)])
    att.kv_append(cache, k, v, slots.to(torch.int32).cuda())
    small = att.KVCache.empty(2, hkv, page, D, BF)
    att.kv_append(small, k, v, torch.arange(n, dtype=torch.int32).cuda())
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    two = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    far = ids[None].cuda()
    assert torch.equal(att.attn_prefill(cache, q, starts, far, lens),
                       att.attn_prefill(small, q, starts, two, lens))
    assert torch.equal(att.attn_decode(cache, q[:4], far, lens),
                       att.attn_decode(small, q[:4], two, lens))


def test_nothing_to_do():
    c = Case([1], [5], 4, 2, 64, BF, BF, 16)
    none = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    table, lens = c.table[:0], torch.empty(0, dtype=torch.int32, device="cuda")
    assert att.attn_decode(c.cache, none, table, lens).shape == (0, 4, 64)
    starts = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert att.attn_prefill(c.cache, none, starts, table, lens).shape == (0, 4, 64)
    q, k = att.qk_norm_rope(none, none, None, att.NormRope())
    assert q.shape == k.shape == (0, 4, 64)
    kv = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    att.kv_append(c.cache, kv, kv, lens)
