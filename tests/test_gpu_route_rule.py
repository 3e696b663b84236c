"""Routing by a rule against a plain 64-bit router, token by token: ids and grouping equal,
weights within half an fp32 step and the last bits of 64-bit sums."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_ref
from quantized_routed_expert_router_amd import qmoe

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _check(logits, k, rule, what=""):
    n, E = logits.shape
    r = qmoe.route_scored(logits, k, rule)
    torch.cuda.synchronize()
    keep = rule.groups if rule.top_groups is None else rule.top_groups
    bias = None if rule.bias is None else rule.bias.cpu().numpy()
    ids, w = mx_ref.route(logits.float().cpu().numpy(), k, rule.score, bias, rule.groups, keep,
                          rule.group_score == "top2", rule.renormalize, rule.scale)
    assert np.array_equal(r.topk_ids.cpu().numpy(), ids), what
    got = r.topk_w.cpu().numpy().astype(np.float64)
    # one rounding to fp32 (2^-24), and 64-bit exponentials, sums and quotients of few roundings;
    # weights below the normal range are off by at most its smallest step
    assert (np.abs(got - w) <= np.abs(w) * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -149).all(), what
    offsets, pairs = mx_ref.grouping(ids, E)
    assert np.array_equal(r.expert_offsets.cpu().numpy(), offsets), what
    assert np.array_equal(r.pair_index.cpu().numpy()[: n * k], pairs), what
    return r


def _logits(n, E, dtype="f32", seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, E), generator=g) * spread).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,E,k,groups,keep", [
    (1, 1, 1, 1, 1), (1, 8, 8, 1, 1), (4, 512, 10, 1, 1), (16, 64, 64, 1, 1), (17, 65, 7, 5, 2),
    (64, 256, 8, 8, 4), (65, 1024, 16, 64, 5), (200, 160, 6, 8, 3), (33, 96, 3, 96 // 2, 7),
    (5, 40, 4, 40, 4), (700, 48, 9, 3, 1), (3, 1024, 64, 1, 1)])
def test_sizes(score, n, E, k, groups, keep):
    groups = min(groups, 64)
    rule = qmoe.RouteRule(score=score, bias=torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() * 0.1,
                          groups=groups, top_groups=keep, group_score="top2", scale=2.5)
    _check(_logits(n, E, seed=n), k, rule)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("pick", ["max", "top2"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_forms(dtype, score, pick, renormalize):
    rule = qmoe.RouteRule(score=score, groups=6, top_groups=4, group_score=pick, renormalize=renormalize)
    _check(_logits(40, 96, dtype, seed=3), 5, rule)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_expert(score):
    # few distinct logits: whole groups and most experts tie, more than 64 at the threshold
    g = torch.Generator().manual_seed(1)
    for E, groups, keep in ((512, 1, 1), (128, 8, 3)):
        logits = torch.randint(-1, 2, (50, E), generator=g).float().cuda()
        logits[0] = 0.0
        logits[1] = -0.0
        for pick in ("max", "top2"):
            _check(logits, 6, qmoe.RouteRule(score=score, groups=groups, top_groups=keep, group_score=pick))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_scores(score):
    # neighbours of one another in fp32: decided by the 64-bit scores
    base = torch.full((40, 128), 0.75)
    steps = torch.randint(-3, 4, (40, 128), generator=torch.Generator().manual_seed(4))
    logits = (base.view(torch.int32) + steps.int()).view(torch.float32).cuda()
    for groups, keep in ((1, 1), (4, 2)):
        _check(logits, 5, qmoe.RouteRule(score=score, groups=groups, top_groups=keep))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n", [3, 30])
def test_masked_rows_and_odd_values(score, n):
    logits = _logits(n, 32, seed=8)
    logits[0] = -torch.inf                      # nothing left: weights 0, experts in order
    logits[1, 3:] = -torch.inf                  # fewer experts than slots
    logits[2, ::2] = torch.finfo(torch.float32).min
    if n > 8:
        logits[3, 5] = torch.nan
        logits[4] = torch.nan
        logits[5, 7] = torch.inf
        logits[6, 7:9] = torch.inf
        logits[7] *= 1e4
    bias = torch.zeros(32).cuda()
    for b in (None, bias, bias.clone().index_fill_(0, torch.tensor([1, 30]).cuda(), -torch.inf),
              bias.clone().index_fill_(0, torch.tensor([2]).cuda(), torch.inf),
              bias.clone().index_fill_(0, torch.tensor([9]).cuda(), torch.nan), bias + 1e6):
        for groups, keep in ((1, 1), (8, 3)):
            r = _check(logits, 6, qmoe.RouteRule(score=score, bias=b, groups=groups, top_groups=keep))
            assert torch.isfinite(r.topk_w).all()


def test_large_logits_keep_their_order_by_id():
    # sigmoid scores of 1 in 64 bits tie
    logits = torch.linspace(30, 60, 64).repeat(2, 1).cuda()
    _check(logits, 8, qmoe.RouteRule())


def test_plain_router_is_the_softmax_rule_without_groups():
    logits = _logits(300, 512, seed=12)
    a = qmoe.route(logits, 10)
    b = qmoe.route_scored(logits, 10, qmoe.RouteRule(score="softmax"))
    assert torch.equal(a.topk_ids, b.topk_ids) and torch.equal(a.pair_index, b.pair_index)
    assert torch.equal(a.expert_offsets, b.expert_offsets)
    assert (a.topk_w - b.topk_w).abs().max() <= 2.0 ** -24  # each within half a step of the same value


def test_no_tokens_and_given_outputs():
    r = qmoe.route_scored(torch.empty((0, 16)).cuda(), 2, qmoe.RouteRule())
    assert r.expert_offsets.tolist() == [0] * 17
    logits = _logits(9, 16)
    out = qmoe.Routing.empty(12, 16, 2)
    out.topk_ids.fill_(-7)
    got = qmoe.route_scored(logits, 2, qmoe.RouteRule(), out=out)
    assert got is out and (out.topk_ids.view(-1)[18:] == -7).all()  # rows behind the last token
    ref = qmoe.route_scored(logits, 2, qmoe.RouteRule())
    assert torch.equal(out.topk_ids.view(-1)[:18], ref.topk_ids.view(-1))


@pytest.mark.parametrize("n", [4, 60, 900])
def test_captured_and_replayed_and_on_another_stream(n):
    rule = qmoe.RouteRule(bias=torch.randn(256).cuda() * 0.1, groups=8, top_groups=4, scale=2.5)
    buf = _logits(n, 256)
    out, ws = qmoe.Routing.empty(n, 256, 8), qmoe.route_workspace(n, 256, 8)
    qmoe.route_scored(buf, 8, rule, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmoe.route_scored(buf, 8, rule, out=out, ws=ws)
    for seed in range(3):
        buf.copy_(_logits(n, 256, seed=seed + 20))
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        ref = qmoe.route_scored(buf, 8, rule, stream=side)
        side.synchronize()
        assert torch.equal(out.topk_ids, ref.topk_ids) and torch.equal(out.topk_w, ref.topk_w)
        assert torch.equal(out.pair_index, ref.pair_index)


def test_refusals():
    x = _logits(4, 32)
    R = qmoe.RouteRule
    for rule, k in ((R(score="tanh"), 2), (R(group_score="mean"), 2)):
        with pytest.raises(ValueError):
            qmoe.route_scored(x, k, rule)
    for rule, k in ((R(groups=5), 2), (R(groups=8, top_groups=9), 2), (R(groups=8, top_groups=0), 2),
                    (R(groups=8, top_groups=1), 5), (R(scale=float("inf")), 2), (R(scale=float("nan")), 2),
                    (R(), 0), (R(), 33), (R(groups=0), 2)):
        with pytest.raises(qmoe.MoeError):
            qmoe.route_scored(x, k, rule)
    for bad in (x.double(), x.t(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            qmoe.route_scored(bad, 2, R())
    with pytest.raises(ValueError):
        qmoe.route_scored(x, 2, R(bias=torch.zeros(31).cuda()))
    with pytest.raises(ValueError):
        qmoe.route_scored(x, 2, R(bias=torch.zeros(32)))
