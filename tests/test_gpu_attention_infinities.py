"""Infinite and NaN values at visible keys whose probability is far below what 16 bits hold:
the row is infinite (NaN), as the formula has it, also in tiles that all rows see."""
from __future__ import annotations

import pytest
import torch

from quantized_routed_expert_router_amd import attention as att

import attn_ref as R

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,gap", [(HF, 20), (HF, 60), (BF, 20), (BF, 95), (HF, 95)])
@pytest.mark.parametrize("D,n,hq,hkv,L", [(64, 5, 4, 2, 500), (128, 33, 4, 1, 500),
                                          (256, 9, 4, 2, 500), (128, 2, 4, 1, 9000),
                                          (64, 2100, 32, 8, 2500), (128, 2100, 32, 8, 2500)])
def test_visible_non_finite_value_of_small_probability(D, n, hq, hkv, L, dtype, gap, value):
    page = 32
    g = torch.Generator().manual_seed(D + n)
    pages = -(-L // page)
    k = torch.zeros((pages, page, hkv, D))
    k[0, 0, :, 0] = gap / 4  # key 0 is gap above all others
    v = torch.randn((pages, page // 8, 8, hkv, D), generator=g)
    v[2, 1, 3, 0, 5] = value  # key 75
    cache = att.KVCache(k.transpose(1, 2).to(dtype).cuda().contiguous(),
                        v.permute(0, 3, 1, 4, 2).to(dtype).cuda().contiguous())
    q = 0.01 * torch.randn((n, hq, D), generator=g)
    q[..., 0] = 4
    q = q.to(dtype).cuda()
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    lens, starts = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([L], [0, n]))
    rows = list(range(n)) if n < 40 else [0, 300, n - 1]
    ref, bound = R.attend(q[rows], (cache.k, cache.v), None, None, table.cpu().expand(len(rows), -1),
                          [L - n + r + 1 for r in rows], list(range(len(rows) + 1)), 1.0, 0, 0, False)
    special = ref[:, : hq // hkv, 5]
    assert (torch.isnan(special) if value != value else special == value).all()
    got = att.attn_prefill(cache, q, starts, table, lens, scale=1.0)
    R.assert_close(got[rows], ref, bound, "prefill")
    # every row sees the key: no other head or column is touched
    hit = torch.zeros((hq, D), dtype=torch.bool)
    hit[: hq // hkv, 5] = True
    assert torch.equal(~torch.isfinite(got).cpu(), hit.expand(n, hq, D))
    if n <= 16:
        R.assert_close(att.attn_decode(cache, q, table, lens, scale=1.0), ref, bound, "decode")
