"""The attention half as it is used: prompt chunks and decode windows through one paged cache,
a decoder layer with its routed experts behind it, captured graphs, streams, and calls side by
side."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import oracle as O
from quantized_routed_expert_router_amd import attention as att
from quantized_routed_expert_router_amd import qmoe, synth, workloads

import attn_ref as R
from gpu_common import assert_output_tolerance, omat, on_side_stream, to_dev

pytestmark = pytest.mark.gpu

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Model:
    """Two sequences' projections, one cache."""

    def __init__(self, lengths, hq=8, hkv=2, D=64, page=16, cdtype=BF, seed=0):
        self.lengths, self.hq, self.hkv, self.D, self.page = lengths, hq, hkv, D, page
        self.qkv = [_rand((n, (hq + 2 * hkv) * D), BF, seed + i) for i, n in enumerate(lengths)]
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + 1
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.table = torch.full((len(lengths), max(need)), -1, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at: at + m]
            at += m
        scale = dict(k_scale=torch.full((hkv,), 0.02).cuda(),
                     v_scale=torch.full((hkv,), 0.02).cuda()) if cdtype == E4 else {}
        self.cache = att.KVCache.empty(pages, hkv, page, D, cdtype, **scale)
        self.p = att.NormRope(1 + _rand((D,), torch.float32, 7, 0.1),
                              1 + _rand((D,), torch.float32, 8, 0.1),
                              (1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()
                              .cuda())

    def heads(self, s, a, b):
        x, hq, hkv, D = self.qkv[s][a:b], self.hq, self.hkv, self.D
        return (x[:, : hq * D].view(-1, hq, D), x[:, hq * D: (hq + hkv) * D].view(-1, hkv, D),
                x[:, (hq + hkv) * D:].view(-1, hkv, D))

    def slots(self, s, a, b):
        pos = torch.arange(a, b)
        return (self.table[s].long()[pos // self.page] * self.page + pos % self.page).to(torch.int32)

    def step(self, spans, attend, **kw):
        """Appends and attends tokens a..b of every sequence; spans: (a, b) of each."""
        parts = [self.heads(s, a, b) for s, (a, b) in enumerate(spans)]
        q, k, v = (torch.cat(x) for x in zip(*parts))
        slots = torch.cat([self.slots(s, a, b) for s, (a, b) in enumerate(spans)]).cuda()
        pos = torch.cat([torch.arange(a, b) for a, b in spans]).to(torch.int32).cuda()
        q = att.kv_append(self.cache, k, v, slots, pos, self.p, q=q)
        lens = _i32([b for _, b in spans])
        if attend == "decode":
            return q, att.attn_decode(self.cache, q, self.table.cuda(), lens, **kw)
        starts = _i32(np.cumsum([0] + [b - a for a, b in spans]).tolist())
        return q, att.attn_prefill(self.cache, q, starts, self.table.cuda(), lens, **kw)


@pytest.mark.parametrize("cdtype,window,sinks", [(BF, 0, 0), (BF, 50, 3), (E4, 0, 0)])
def test_prompt_then_decode(cdtype, window, sinks):
    # uneven prompt chunks, then verify windows of 4 and single tokens; every output against
    # the 64-bit attention over what the cache holds at the end (causal: later rows do not
    # matter to earlier tokens)
    m = Model([230, 161], cdtype=cdtype)
    plan = [("prefill", [(0, 101), (0, 37)]), ("prefill", [(101, 205), (37, 120)]),
            ("decode", [(205, 209), (120, 124)]), ("decode", [(209, 213), (124, 128)]),
            ("decode", [(213, 214), (128, 129)]), ("prefill", [(214, 230), (129, 161)])]
    got = []
    for kind, spans in plan:
        q, out = m.step(spans, kind, window=window, sinks=sinks)
        got.append((kind, spans, q, out))
    # what the cache holds is the normed and rotated keys, and the values
    for s, n in enumerate(m.lengths):
        _, k, v = m.heads(s, 0, n)
        ref = R.norm_rope(k, m.p.k_norm, torch.arange(n), m.p.inv_freq, 1e-6)
        held_k, held_v, _ = R.gather((m.cache.k, m.cache.v), m.cache.k_scale, m.cache.v_scale,
                                     m.table[s], n)
        if cdtype == BF:
            R.assert_close(held_k.transpose(0, 1), ref, R.rows_bound(ref, BF), "keys")
            assert torch.equal(held_v.transpose(0, 1), v.double().cpu())
        else:
            step = 0.02 * (2.0 ** -10) + 2.0 ** -4 * ref.abs() * 1.01 + 2.0 ** -20 * 16
            R.assert_close(held_k.transpose(0, 1), ref, step, "8-bit keys")
    for kind, spans, q, out in got:
        starts = np.cumsum([0] + [b - a for a, b in spans]).tolist()
        ref, bound = R.attend(q, (m.cache.k, m.cache.v), m.cache.k_scale, m.cache.v_scale, m.table,
                              [b for _, b in spans], starts, 1 / math.sqrt(m.D), window, sinks,
                              kind == "decode")
        R.assert_close(out, ref, bound, f"{kind} {spans}")


def test_decoder_layer():
    # one decoder layer of a verify window: attention half, output projection into the
    # residual, routed experts behind it (shape of the smallest layer: 256 wide, 8 experts)
    w = synth.Workload("layer", 256, 128, 8, 2, 4, 4, "normal")
    host = synth.host_layer(w, 0)
    layer = workloads.layer_from_host(*host, w.k)
    m = Model([64], hq=4, hkv=2, D=64)
    m.step([(0, 60)], "prefill")
    lg, x = synth.layer_inputs(w, 0)
    residual = to_dev(x)
    q, out = m.step([(60, 64)], "decode")
    ref, bound = R.attend(q, (m.cache.k, m.cache.v), None, None, m.table, [64], [0, 4], 0.125, 0, 0,
                          True)
    R.assert_close(out, ref, bound, "attention")
    wo = _rand((256, 256), BF, 21, 1 / 16)
    residual += (out.reshape(4, 256).float() @ wo.float())
    before = residual.cpu().numpy()
    r = qmoe.layer_decode(layer, to_dev(lg), residual, residual)
    torch.cuda.synchronize()
    ids, wt = O.route(lg, w.k)
    assert np.array_equal(r.topk_ids.cpu().numpy(), ids)
    want, _ = O.ffn_decode(*(omat(h) for h in host), w.E, before, ids, wt, before)
    assert_output_tolerance(residual.cpu().numpy(), want)
    assert_output_tolerance(residual.cpu().numpy() - before, want - before, what="moe delta")


@pytest.mark.parametrize("D,cdtype,long", [(64, BF, 300), (128, E4, 300), (64, BF, 5000)])
def test_graph_replays(D, cdtype, long):
    # append + decode attention (with its joining launch at the long context) + a routed layer
    # captured once; replayed as the sequence grows, positions, slots and lengths updated in
    # place between replays; every replay bit-identical to the eager calls
    w = synth.Workload("layer", 512, 256, 16, 4, 4, 4, "normal")
    layer = workloads.layer_from_host(*synth.host_layer(w, 0), w.k)
    lg, x = (to_dev(a) for a in synth.layer_inputs(w, 0))
    first = long - 4 * 4
    eager, graph = (Model([long], hq=8, hkv=2, D=D, cdtype=cdtype) for _ in range(2))
    for m in (eager, graph):
        m.cache.k.view(torch.uint8).zero_()
        m.cache.v.view(torch.uint8).zero_()
        for a in range(0, first, 4096):
            m.step([(a, min(a + 4096, first))], "prefill")
    table = graph.table.cuda()
    ws_bytes = att.decode_workspace_bytes(graph.cache, 8, 1, 4, table.shape[1])
    assert (ws_bytes > 0) == (long > 1000)
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device="cuda")
    q_in, k_in, v_in = (t.clone() for t in graph.heads(0, first, first + 4))
    slots, pos, lens = graph.slots(0, first, first + 4).cuda(), _i32(range(4)), _i32([0])
    q_out, out = torch.empty_like(q_in), torch.empty_like(q_in)
    res = torch.empty_like(x)
    routing = qmoe.Routing.empty(4, w.E, w.k)
    lws = qmoe.workspace(layer, 4)

    def body():
        att.kv_append(graph.cache, k_in, v_in, slots, pos, graph.p, q=q_in, q_out=q_out)
        att.attn_decode(graph.cache, q_out, table, lens, out=out, ws=ws)
        res.copy_(x)
        qmoe.layer_decode(layer, lg, res, res, routing=routing, ws=lws)

    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        body()
    torch.cuda.synchronize()
    res_e = x.clone()
    qmoe.layer_decode(layer, lg, res_e, res_e)
    for step in range(4):
        a = first + 4 * step
        for dst, src in zip((q_in, k_in, v_in), graph.heads(0, a, a + 4)):
            dst.copy_(src)
        slots.copy_(graph.slots(0, a, a + 4))
        pos.copy_(torch.arange(a, a + 4, dtype=torch.int32))
        lens.fill_(a + 4)
        out.fill_(-1)
        ws.fill_(0xff)  # the workspace needs no contents
        (torch.randn(1 << 14, device="cuda") * 2).sum().item()
        g.replay()
        torch.cuda.synchronize()
        q_e, out_e = eager.step([(a, a + 4)], "decode")
        assert torch.equal(q_out, q_e) and torch.equal(out, out_e), f"replay {step}"
        for x_, y_ in ((graph.cache.k, eager.cache.k), (graph.cache.v, eager.cache.v)):
            assert torch.equal(x_.view(torch.uint8), y_.view(torch.uint8)), f"replay {step}: cache"
        assert torch.equal(res, res_e), f"replay {step}: experts"


def test_prefill_graph_replays():
    m = Model([700, 90])
    want = [m.step([(0, 650), (0, 90)], "prefill")[1], m.step([(650, 700), (80, 90)], "prefill")[1]]
    table, lens = m.table.cuda(), _i32([700, 90])
    starts = _i32([0, 50, 60])
    parts = [m.heads(0, 650, 700)[0], m.heads(1, 80, 90)[0]]
    pos = torch.cat([torch.arange(650, 700), torch.arange(80, 90)]).to(torch.int32).cuda()
    q, _ = att.qk_norm_rope(torch.cat(parts), None, pos, m.p)
    out = torch.empty_like(q)
    ws = torch.empty(max(256, att.prefill_workspace_bytes(m.cache, 8, 2, 60, table.shape[1])),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        att.attn_prefill(m.cache, q, starts, table, lens, out=out, ws=ws)
    for rep in range(3):
        out.fill_(5)
        ws.fill_(0xff)
        (torch.randn(1 << 14, device="cuda") * 2).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[1]), f"replay {rep}"


def test_calls_follow_the_current_stream():
    # inputs that arrive behind a spin on a side stream: every launch is on that stream
    m = Model([400])
    q, k, v = m.heads(0, 0, 400)
    slots, pos = m.slots(0, 0, 400).cuda(), torch.arange(400, dtype=torch.int32).cuda()
    table, lens, starts = m.table.cuda(), _i32([400]), _i32([0, 400])
    want_q = att.kv_append(m.cache, k, v, slots, pos, m.p, q=q)
    want = att.attn_prefill(m.cache, want_q, starts, table, lens)
    want_d = att.attn_decode(m.cache, want_q[-4:].contiguous(), table, lens)
    torch.cuda.synchronize()
    ck, cv = m.cache.k.clone(), m.cache.v.clone()
    m.cache.k.zero_()
    m.cache.v.zero_()
    torch.cuda.synchronize()

    def call(qs, ks, vs):
        c = att.KVCache(m.cache.k, m.cache.v)
        qo = att.kv_append(c, ks, vs, slots, pos, m.p, q=qs)
        return (att.attn_prefill(c, qo, starts, table, lens),
                att.attn_decode(c, qo[-4:].contiguous(), table, lens))

    _, (got, got_d) = on_side_stream([q.contiguous(), k.contiguous(), v.contiguous()], call)
    assert torch.equal(got, want) and torch.equal(got_d, want_d)
    live = m.table[0].long()[torch.arange(400) // m.page] * m.page + torch.arange(400) % m.page
    at = live.cuda()
    assert torch.equal(m.cache.k[at // m.page, :, at % m.page], ck[at // m.page, :, at % m.page])
    assert torch.equal(m.cache.v[at // m.page, :, at % m.page // 8, :, at % 8],
                       cv[at // m.page, :, at % m.page // 8, :, at % 8])


def test_stream_argument_and_two_calls_at_once():
    # two decode calls with split keys on two streams at once, workspaces of their own; what
    # they return is used on the default stream afterwards
    m = Model([6000, 6000], seed=4)
    for a in (0, 4000):
        m.step([(a, a + 2000), (a, a + 2000)], "prefill")
    m.step([(2000, 4000), (2000, 4000)], "prefill")
    table = m.table.cuda()
    qs = [_rand((4, 8, 64), BF, 30 + s) for s in range(2)]
    want = [att.attn_decode(m.cache, qs[s], table[s: s + 1], _i32([6000])) for s in range(2)]
    lens = _i32([6000])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(3):
        got = [att.attn_decode(m.cache, qs[s], table[s: s + 1], lens, stream=streams[s])
               for s in range(2)]
        junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"round {rep}"
        del junk


def test_short_path_and_checked_path_agree():
    # the same call with and without given outputs takes the two marshalling paths
    m = Model([90])
    q, k, v = m.heads(0, 0, 90)
    slots, pos = m.slots(0, 0, 90).cuda(), torch.arange(90, dtype=torch.int32).cuda()
    a = att.kv_append(m.cache, k, v, slots, pos, m.p, q=q)
    b = torch.empty_like(a)
    assert att.kv_append(m.cache, k, v, slots, pos, m.p, q=q, q_out=b) is b
    assert torch.equal(a, b)
    qa, ka = att.qk_norm_rope(q, k, pos, m.p)
    qb, kb = att.qk_norm_rope(q, k, pos, m.p, q_out=torch.empty_like(qa))
    assert torch.equal(qa, qb) and torch.equal(ka, kb) and torch.equal(qa, a)
    table, lens, starts = m.table.cuda(), _i32([90]), _i32([0, 90])
    for fn, args in ((att.attn_decode, (m.cache, a[-2:], table, lens)),
                     (att.attn_prefill, (m.cache, a, starts, table, lens))):
        x = fn(*args)
        y = fn(*args, out=torch.empty_like(x))
        assert torch.equal(x, y)
    with pytest.raises(qmoe.MoeError) as e:
        att.attn_decode(m.cache, torch.zeros((17, 8, 64), dtype=BF, device="cuda"), table, lens)
    assert e.value.status == 1
    with pytest.raises(qmoe.MoeError) as e:
        att.attn_decode(m.cache, torch.zeros((1, 8, 64), dtype=torch.float16, device="cuda"), table,
                        lens)
    assert e.value.status == 2
    with pytest.raises(ValueError, match="page_table: dtype"):
        att.attn_decode(m.cache, a[-2:], table.long(), lens)
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        att.attn_decode(m.cache, a[-2:], table.cpu(), lens)
    with pytest.raises(ValueError, match="window, sinks"):
        att.attn_decode(m.cache, a[-2:], table, lens, window=-3)
