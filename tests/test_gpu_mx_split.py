"""Every tile of the grouped products is computed, whatever the numbers of pairs an expert: the
workspace holds NaN before the call, and a row that no workgroup wrote would stay NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_ref
from quantized_routed_expert_router_amd import mx, qmoe

pytestmark = pytest.mark.gpu


def _layer(E, d, f, k, seed):
    def weights(rows, cols, s):
        return mx.quantize((torch.randn((E, rows, cols), generator=torch.Generator().manual_seed(s)) * 0.02).cuda())
    return mx.MxLayer(weights(f, d, seed), weights(f, d, seed + 1), weights(d, f, seed + 2), k)


def _ids(kind, n, E, k, rng):
    if kind == "one":
        return np.full((n, k), E // 2)
    if kind == "even":
        return np.arange(n * k).reshape(n, k) % E
    if kind == "few":  # most pairs to a few experts, the rest anywhere
        few = rng.integers(0, E, (n, k)) % max(1, E // 50)
        return np.where(rng.random((n, k)) < 0.9, few, rng.integers(0, E, (n, k)))
    return (E * rng.random((n, k)) ** 4).astype(np.int64)


@pytest.mark.parametrize("kind", ["one", "even", "few", "skewed"])
@pytest.mark.parametrize("n,E,k,d,f", [(17, 1024, 4, 64, 32), (300, 3, 2, 320, 160), (1000, 1024, 6, 64, 32),
                                       (2111, 64, 8, 64, 288), (8192, 300, 4, 64, 32)])
def test_all_tiles(kind, n, E, k, d, f):
    rng = np.random.default_rng(n + E)
    ids = _ids(kind, n, E, k, rng).astype(np.int32)
    offsets, pairs = mx_ref.grouping(ids, E)
    layer = _layer(E, d, f, k, seed=n)
    x = torch.randn((n, d), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.rand((n, k), generator=torch.Generator().manual_seed(2)).cuda()
    r = qmoe.Routing(*(torch.from_numpy(a).cuda() if isinstance(a, np.ndarray) else a for a in (ids, w, offsets, pairs)))
    ws = torch.full((mx.ffn_workspace_bytes(layer, n),), 0xff, dtype=torch.uint8, device="cuda")
    out = mx.ffn(layer, x, r, ws=ws)
    assert torch.isfinite(out).all()
    t = torch.from_numpy(rng.integers(0, n, 8))
    ref, bound = mx_ref.ffn(layer, x[t.cuda()], r.topk_ids[t.cuda()].long(), w[t.cuda()], torch.zeros((8, d)).cuda())
    assert ((out[t.cuda()].double() - ref).abs() <= bound).all()
