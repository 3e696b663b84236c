"""Routing records of a shard of the experts: what the slots of other shards' pairs hold, their
weights among it, does not reach the output."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_ref
from quantized_routed_expert_router_amd import mx, qmoe

pytestmark = pytest.mark.gpu

E, K, D, F = 6, 4, 128, 64


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _layer(seed):
    def weights(rows, cols, s):
        return mx.quantize((torch.randn((E, rows, cols), generator=_gen(s)) * 0.02).cuda())
    return mx.MxLayer(weights(F, D, seed), weights(F, D, seed + 1), weights(D, F, seed + 2), K)


def _record(ids, w):
    """Groups that hold the pairs of experts 0..E-1 alone."""
    flat = ids.view(-1).numpy()
    pairs = np.argsort(flat, kind="stable")
    pairs = pairs[(flat[pairs] >= 0) & (flat[pairs] < E)]
    offsets = np.concatenate(([0], np.bincount(flat[pairs], minlength=E).cumsum())).astype(np.int32)
    pairs = np.concatenate((pairs, np.zeros(ids.numel() - len(pairs)))).astype(np.int32)
    return qmoe.Routing(ids.cuda(), w.cuda(), torch.from_numpy(offsets).cuda(), torch.from_numpy(pairs).cuda())


@pytest.mark.parametrize("n", [1, 3, 16, 17, 40, 300])  # the window up to 16 tokens, grouped above
@pytest.mark.parametrize("odd", [torch.nan, torch.inf, -torch.inf])
def test_weights_of_pairs_of_no_expert_are_not_read(n, odd):
    layer = _layer(17)
    x = torch.randn((n, D), generator=_gen(18)).bfloat16().cuda()
    residual = torch.randn((n, D), generator=_gen(19)).cuda()
    ids = torch.randint(0, E, (n, K), generator=_gen(20), dtype=torch.int32)
    drop = torch.rand((n, K), generator=_gen(21)) < 0.4
    drop[0] = True
    ids[drop] = torch.where(torch.rand(int(drop.sum()), generator=_gen(22)) < 0.5, -1, E).int()
    w = torch.rand((n, K), generator=_gen(23))
    plain = mx.ffn(layer, x, _record(ids, w), residual)
    w[drop] = odd
    r = _record(ids, w)
    out = mx.ffn(layer, x, r, residual)
    assert torch.isfinite(out).all()
    assert torch.equal(out, plain) and torch.equal(out[0], residual[0])
    # the sums' roundings are bounded there; pairs of no expert take no part in it
    ref, bound = mx_ref.ffn(layer, x, ids.long().cuda(), r.topk_w, residual)
    assert ((out.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("n", [4, 40])
def test_weights_of_experts_are_read_whatever_they_are(n):
    layer = _layer(27)
    x, residual = torch.randn((n, D), generator=_gen(28)).cuda(), torch.zeros((n, D)).cuda()
    ids = torch.randint(0, E, (n, K), generator=_gen(29), dtype=torch.int32)
    w = torch.rand((n, K), generator=_gen(30))
    w[1, 2] = torch.nan
    out = mx.ffn(layer, x, _record(ids, w), residual)
    rest = torch.arange(n) != 1
    assert out[1].isnan().all() and torch.isfinite(out[rest.cuda()]).all()
