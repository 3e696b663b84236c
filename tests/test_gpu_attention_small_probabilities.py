"""Attention rows with one dominant key and a long tail of small probabilities, in fp16.

The dominant keys' values are 0, so the output is the tail's part alone: what the 16-bit
probabilities of the second product lose of it shows in full.

The tolerance, row by row, with p the probabilities (relative to the row's sum) and v the
values in fp16:
* rounding of the output: half a step, 2^-11 |o|, or 2^-25 below 2^-14;
* rounding of a probability to fp16: 2^-11 p in prefill; in decode the value and its rest
  leave 2^-22 p;
* a probability below the smallest normal number, 2^-14, is off by at most 2^-25 instead. The
  kernels hold probabilities times 2^11, the dominant key's (the row's largest) at no less
  than 2^11, so with `tops` equal dominant keys the L keys together are off by at most
  2^-36 L / tops of the largest value, against the row's sum;
* scores in fp32: D products and sums of at most sum |q||k|, in the exponent of the numerator and
  of the denominator; fp32 sums over L keys, exp2, scaling and division: 2^-24 (2 (D + 8) sum
  |q||k| + L + 32), relative to sum p |v|.
"""
from __future__ import annotations

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

import attn_ref as R

pytestmark = pytest.mark.gpu

HF, E4 = torch.float16, torch.float8_e4m3fn


class Tail:
    """One sequence of L keys in shuffled pages: `every` == 0: key 0 dominates, else every
    32nd key, by `gap` in the exponent."""

    def __init__(self, n, L, hq, hkv, D, gap, every, cdtype=HF, page=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        pages = -(-L // page) + 1
        at = torch.arange(L)
        top = at % 32 == every - 1 if every else at == 0
        k = 0.25 * torch.randn((L, hkv, D), generator=g)
        v = (300 + 60 * torch.randn((L, hkv, D), generator=g)).clamp(100, 440)
        k[..., 0] = 0
        k[top] = 0
        k[..., 0][top] = gap / 4
        v[top] = 0
        self.tops = (L - n) // 32 if every else 1  # as many as every row sees at least
        q = 0.25 * torch.randn((n, hq, D), generator=g)
        q[..., 0] = 4
        ck, cv = torch.zeros((pages, hkv, page, D)), torch.zeros((pages, hkv, page, D))
        order = torch.randperm(pages, generator=g)[: -(-L // page)]
        ck[order[at // page], :, at % page] = k
        cv[order[at // page], :, at % page] = v
        cv = cv.view(pages, hkv, page // 8, 8, D).transpose(3, 4).contiguous()
        self.scales = (None, None)
        if cdtype == E4:
            self.scales = (torch.full((hkv,), 0.03125).cuda(), torch.ones(hkv).cuda())
            ck = ck * 32
        self.cache = att.KVCache(ck.to(cdtype).cuda(), cv.to(cdtype).cuda(), *self.scales)
        self.q, self.L = q.to(HF).cuda(), L
        self.table = order[None].to(torch.int32).cuda()

    def check(self, got, rows, part, what):
        """got [n, hq, D] against 64 bits at the tokens `rows` (the last token sees L keys)."""
        n, hq, D = self.q.shape
        rows = sorted(set(r % n for r in rows))
        lens = [self.L - n + r + 1 for r in rows]
        q = self.q[rows]
        ref, _ = R.attend(q, (self.cache.k, self.cache.v), *self.scales,
                          self.table.cpu().expand(len(rows), -1), lens, list(range(len(rows) + 1)),
                          1.0, 0, 0, False)
        k, v, _ = R.gather((self.cache.k, self.cache.v), *self.scales, self.table[0], self.L)
        # all values are of one sign: sum p |v| is the output itself
        assert (v >= 0).all() and (ref > 0).all()
        big = max(float((q[:, h].double().cpu().abs() @ k[h // (hq // k.shape[0])].abs().T).amax())
                  for h in range(hq))
        slack = part + 2.0 ** -24 * (2 * (D + 8) * big + self.L + 32)
        least = 2.0 ** -36 * self.L / self.tops * float(v.amax())
        bound = (2.0 ** -11 * 1.01 + slack) * ref + least + 2.0 ** -25
        # the tolerance leaves no room for a lost tail
        assert float((bound / ref).amax()) < 0.2
        R.assert_close(got[rows], ref, bound, what)


@pytest.mark.parametrize("gap", [14, 16, 17, 18])
@pytest.mark.parametrize("D,hq,hkv,n,cdtype", [(64, 8, 2, 5, HF), (128, 4, 1, 40, HF),
                                               (256, 4, 2, 7, HF), (128, 4, 2, 9, E4)])
def test_prefill_tail(D, hq, hkv, n, cdtype, gap):
    c = Tail(n, 700, hq, hkv, D, gap, 32, cdtype)
    got = att.attn_prefill(c.cache, c.q, torch.tensor([0, n], dtype=torch.int32).cuda(), c.table,
                           torch.tensor([700], dtype=torch.int32).cuda(), scale=1.0)
    c.check(got, range(n), 2.0 ** -11, f"prefill, gap {gap}")


@pytest.mark.parametrize("gap", [17, 18])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_tail_behind_a_first_key(D, gap):
    # 8 waves a workgroup, which take the whole context in one piece
    n, L = 2100, 40000
    c = Tail(n, L, 32, 8, D, gap, 0)
    assert att.prefill_workspace_bytes(c.cache, 32, 1, n, c.table.shape[1]) == 0
    got = att.attn_prefill(c.cache, c.q, torch.tensor([0, n], dtype=torch.int32).cuda(), c.table,
                           torch.tensor([L], dtype=torch.int32).cuda(), scale=1.0)
    c.check(got, [0, 777, n - 1], 2.0 ** -11, f"prefill, gap {gap}")


@pytest.mark.parametrize("gap", [8, 14, 17, 18])
@pytest.mark.parametrize("D,hq,hkv,n,L,cdtype", [
    (64, 8, 2, 1, 700, HF), (64, 40, 1, 2, 700, HF), (128, 4, 2, 4, 900, HF), (256, 8, 1, 5, 700, HF),
    (128, 16, 1, 4, 900, E4), (128, 8, 2, 2, 9000, HF),  # the last one with joined splits
])
def test_decode_tail(D, hq, hkv, n, L, cdtype, gap):
    c = Tail(n, L, hq, hkv, D, gap, 32, cdtype)
    got = att.attn_decode(c.cache, c.q, c.table, torch.tensor([L], dtype=torch.int32).cuda(),
                          scale=1.0)
    c.check(got, range(n), 2.0 ** -22, f"decode, gap {gap}")
