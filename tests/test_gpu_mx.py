"""Microscaled 4-bit quantization and products against their definitions in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_ref
from quantized_routed_expert_router_amd import mx, qmoe

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(shape, dtype="bf16", seed=0, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * scale).to(TYPES[dtype]).cuda()


def _same_codes(x, m):
    code, scale = mx_ref.quantize(x.double().cpu().numpy())
    assert np.array_equal(m.scales.cpu().numpy(), scale)
    got, ref = m.codes.cpu().numpy(), mx_ref.pack(code)
    assert np.array_equal(got, ref)


# ---------------------------------------------------------------- quantization


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 32), (1, 96), (7, 2080), (513, 64), (2, 3, 160), (40, 8192)])
def test_quantize_sizes(dtype, shape):
    x = _normal(shape, dtype, seed=sum(shape), scale=3.0)
    _same_codes(x, mx.quantize(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_16_bit_pattern(dtype):
    # each pattern beside larger ones of every exponent, infinities and NaN among them
    bits = torch.arange(1 << 16, dtype=torch.int32)
    for other in range(0, 16):
        x = torch.empty((1 << 16, 32), dtype=torch.int32)
        x[:] = bits[:, None]
        x[:, 1::2] = ((bits + (other << 7 if dtype == "bf16" else other << 10)) & 0xFFFF)[:, None]
        v = x.to(torch.int16).view(TYPES[dtype]).cuda()
        _same_codes(v, mx.quantize(v))


def test_quantize_f32_borders_and_ends():
    near = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999, 4.0, 1.0, 0.5, 0.0])
    steps = torch.cat([near, torch.nextafter(near, torch.tensor(10.0)), torch.nextafter(near, torch.tensor(-10.0))])
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -124, -120, -1, 0, 1, 60, 120, 124, 125):
        for top in (4.0, 7.99, 1.0, 5.0):
            for i in range(0, len(steps), 14):
                r = torch.zeros(32, dtype=torch.float64)
                r[:14] = steps[i: i + 14].double()
                r[14:28] = -steps[i: i + 14].double()
                r[28] = top
                rows.append((r * 2.0 ** e).clamp(-3.4e38, 3.4e38).float())
    x = torch.stack(rows).cuda()
    _same_codes(x, mx.quantize(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_odd_values(dtype):
    x = _normal((8, 96), dtype, seed=2)
    x[1] = 0
    x[2] = -0.0
    x[3, 40] = torch.inf
    x[4, 95] = torch.nan
    x[5, :32] = -torch.inf
    x[6] = torch.finfo(TYPES[dtype]).max
    x[7] = torch.finfo(TYPES[dtype]).smallest_normal
    m = mx.quantize(x)
    _same_codes(x, m)
    v = mx.dequantize(m)
    ref = mx_ref.values(m.codes.cpu().numpy(), m.scales.cpu().numpy()).astype(np.float32)
    assert np.array_equal(v.cpu().numpy(), ref, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_dequantize_every_code_and_scale(dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).reshape(256, 256)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    m = mx.MxMatrix(codes.cuda(), scales.cuda())
    got = mx.dequantize(m, TYPES[dtype])
    ref = torch.from_numpy(mx_ref.values(codes.numpy(), scales.numpy())).float().to(TYPES[dtype])
    assert torch.equal(torch.nan_to_num(got.cpu(), nan=-1.0), torch.nan_to_num(ref, nan=-1.0))
    assert torch.equal(got.isnan().cpu(), ref.isnan())


def test_quantize_strided_rows_and_neighbours():
    big = _normal((50, 6, 64), "bf16", seed=5)
    view = big[:, 2]  # row stride 384
    out = mx.MxMatrix.empty(50, 64)
    guard = mx.MxMatrix(torch.full((52, 32), 9, dtype=torch.uint8).cuda(), torch.full((52, 2), 9, dtype=torch.uint8).cuda())
    _same_codes(view, mx.quantize(view))
    _same_codes(view, mx.quantize(view, out=out))
    inner = mx.MxMatrix(guard.codes[:50], guard.scales[:50])
    mx.quantize(view, out=inner)
    assert (guard.codes[50:] == 9).all() and (guard.scales[50:] == 9).all()
    empty = mx.quantize(big[:0, 2])
    assert empty.codes.shape == (0, 32) and mx.dequantize(empty).shape == (0, 64)


# ---------------------------------------------------------------- linear


def _weights(rows, cols, seed):
    """4-bit normal weights; blocks' exponents within a few of each other."""
    return mx.quantize(_normal((rows, cols), "f32", seed, 0.02))


def _check_linear(x, w, got, quantized=None):
    q = mx_ref.rounded(x) if quantized is None else mx_ref.matrix(quantized)
    wv = mx_ref.matrix(w)
    ref = q @ wv.T
    size = q.abs() @ wv.abs().T
    # at most K / 64 + 4 fp32 additions of exact block sums, then one rounding to the type
    steps = x.shape[1] / 64 + 4 if x is not None else q.shape[1] / 64 + 4
    half = torch.finfo(got.dtype).eps / 2
    bound = size * steps * 2.0 ** -24 + ref.abs() * half + torch.finfo(got.dtype).smallest_normal * half
    assert ((got.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("n,K,N", [
    (1, 32, 1), (1, 2048, 5120), (4, 2080, 33), (16, 8192, 40), (17, 128, 128), (17, 32, 3), (3, 9216, 50),
    (5, 160, 31), (64, 96, 64), (65, 512, 129), (200, 1056, 300), (517, 2080, 1441), (130, 4096, 257),
    (1025, 608, 1300), (1100, 512, 1024), (2000, 256, 777), (300, 2880, 4500), (1, 64, 1), (40, 32, 7), (40, 64, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_sizes(n, K, N, dtype):
    x, w = _normal((n, K), dtype, seed=n + K), _weights(N, K, seed=N)
    _check_linear(x, w, mx.linear(x, w))
    for out in ("f32", "bf16"):
        _check_linear(x, w, mx.linear(x, w, dtype=TYPES[out]))
    q = mx.quantize(x)
    a, b = mx.linear(q, w, dtype=torch.float32), mx.linear(x, w, dtype=torch.float32)
    assert torch.equal(a, b)  # one quantization for several products


@pytest.mark.parametrize("n", [2, 40, 1500])
@pytest.mark.parametrize("K", [96, 512, 1088])
def test_linear_strides_and_neighbours(n, K):
    N = 72
    x = _normal((n, K + 64), "bf16", seed=3)[:, 32: 32 + K]
    w = _weights(N, K, seed=4)
    frame = torch.full((n + 2, N + 9), 7.0).cuda()
    out = frame[1: n + 1, 3: 3 + N]
    assert mx.linear(x, w, out=out) is out
    _check_linear(x, w, out)
    out.fill_(7.0)
    assert (frame == 7.0).all()  # nothing around it was written


@pytest.mark.parametrize("n,K,N", [(3, 96, 40), (70, 160, 90), (1100, 1024, 1030)])
def test_linear_nan_blocks_and_wide_scales(n, K, N):
    x = _normal((n, K), "f32", seed=6)
    x *= torch.exp2(torch.randint(-40, 40, (n, K // 32), generator=_gen(7)).float()).repeat_interleave(32, 1).cuda()
    w = _weights(N, K, seed=8)
    w.scales += torch.randint(0, 30, w.scales.shape, generator=_gen(9), dtype=torch.uint8).cuda()
    _check_linear(x, w, mx.linear(x, w))
    x[1, K - 5] = torch.inf
    w.scales[2, 0] = 255
    w.scales[N - 1, -1] = 255
    got = mx.linear(x, w)
    assert got[1].isnan().all() and got[:, 2].isnan().all() and got[:, N - 1].isnan().all()
    fine = got.isnan()
    fine[1], fine[:, 2], fine[:, N - 1] = False, False, False
    assert not fine.any()


@pytest.mark.parametrize("n", [1, 9, 200])
def test_linear_into_given_rows_and_of_quantized_rows(n):
    w, x = _weights(72, 160, 3), _normal((n, 160), "bf16", seed=n)
    q = mx.quantize(x)
    for dtype in TYPES.values():
        ref = mx.linear(x, w, dtype=dtype)
        frame = torch.full((n + 1, 80), 5.0, dtype=dtype).cuda()
        out = frame[:n, :72]
        assert mx.linear(x, w, out=out) is out and torch.equal(out, ref)
        out.zero_()
        assert mx.linear(q, w, out=out) is out and torch.equal(out, ref)
        assert torch.equal(mx.linear(q, w, dtype=dtype), ref)
        assert (frame[n:] == 5).all() and (frame[:, 72:] == 5).all()
    for bad in (torch.empty((n + 1, 72)), torch.empty((n, 71)), torch.empty((n, 72), dtype=torch.float64)):
        with pytest.raises(ValueError):
            mx.linear(q, w, out=bad.cuda())
    with pytest.raises(ValueError):
        mx.linear(x, w, out=torch.empty((n, 72)).cuda(), dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.linear(mx.quantize(_normal((n, 128))), w)


def test_linear_at_the_end_of_its_memory():
    # the last scales are read in whole requests: nothing behind them is, wherever they end
    for n, K, N in ((20, 32, 16), (33, 32, 17), (33, 64, 9), (64, 96, 19), (40, 288, 21), (1200, 416, 1001)):
        w = _weights(N, K, seed=N)
        size = w.scales.numel()
        arena = torch.full((size + 4096,), 255, dtype=torch.uint8).cuda()
        at = (4096 - size) % 16 if size < 4096 else 0
        at = at - at % 16
        arena[at: at + size] = w.scales.view(-1)
        placed = mx.MxMatrix(w.codes, arena[at: at + size].view(N, K // 32))
        x = _normal((n, K), "bf16", seed=n)
        _check_linear(x, w, mx.linear(x, placed))  # the bytes around are NaN scales


# ---------------------------------------------------------------- routed experts


def _layer(E, d, f, k, seed=0):
    return mx.MxLayer(mx.MxMatrix(*_split(_weights(E * f, d, seed), E)),
                      mx.MxMatrix(*_split(_weights(E * f, d, seed + 1), E)),
                      mx.MxMatrix(*_split(_weights(E * d, f, seed + 2), E)), k)


def _split(m, E):
    return m.codes.view(E, -1, m.codes.shape[1]), m.scales.view(E, -1, m.scales.shape[1])


def _routing(n, E, k, seed=0, skew=0.0):
    logits = torch.randn((n, E), generator=_gen(seed)) - skew * torch.arange(E).float()
    return qmoe.route(logits.cuda(), k)


def _check_ffn(layer, x, r, residual, out):
    n, k = x.shape[0], layer.top_k
    res = torch.zeros_like(out) if residual is None else residual
    ids = r.topk_ids.view(-1)[: n * k].view(n, k).long()
    ref, bound = mx_ref.ffn(layer, x, ids, r.topk_w.view(-1)[: n * k].view(n, k), res)
    assert ((out.double() - ref).abs() <= bound + 1e-37).all(), ((out.double() - ref).abs() / bound.clamp(min=1e-37)).max()


@pytest.mark.parametrize("n,E,k,d,f", [
    (1, 1, 1, 32, 32), (1, 8, 2, 256, 128), (4, 16, 4, 160, 96), (16, 40, 16, 128, 64), (16, 64, 10, 2048, 768),
    (17, 8, 2, 256, 256), (40, 8, 3, 96, 32), (5, 64, 64, 32, 32), (130, 4, 2, 384, 160), (300, 16, 4, 544, 288),
    (33, 3, 3, 2080, 96), (256, 64, 8, 512, 512), (9, 7, 5, 8192, 32), (20, 5, 2, 64, 1056)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_sizes(n, E, k, d, f, dtype):
    layer = _layer(E, d, f, k, seed=E)
    x = _normal((n, d), dtype, seed=n)
    r = _routing(n, E, k, seed=d)
    residual = _normal((n, d), "f32", seed=f)
    out = mx.ffn(layer, x, r, residual)
    _check_ffn(layer, x, r, residual, out)
    again = mx.ffn(layer, x, r, residual)
    assert torch.equal(out, again)
    assert torch.equal(mx.ffn(layer, x, r), mx.ffn(layer, x, r, torch.zeros_like(residual)))
    kept = residual.clone()
    assert mx.ffn(layer, x, r, kept, out=kept) is kept and torch.equal(kept, out)


@pytest.mark.parametrize("n", [3, 16, 200, 600])
def test_ffn_uneven_experts(n):
    # one expert takes nearly all rows, some none, some a few
    layer = _layer(24, 256, 128, 4, seed=3)
    x, residual = _normal((n, 256), "f16", seed=1), _normal((n, 256), "f32", seed=2)
    r = _routing(n, 24, 4, seed=5, skew=0.5)
    assert (r.expert_offsets[1:] == r.expert_offsets[:-1]).any()
    _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))


@pytest.mark.parametrize("n", [1, 5, 6, 16])
def test_ffn_few_large_experts(n):
    # few tokens whose pairs read the same large experts: on both sides of the window's end
    layer = _layer(2, 2048, 4096, 2, seed=41)
    x, residual = _normal((n, 2048), "bf16", seed=n), _normal((n, 2048), "f32", seed=42)
    r = _routing(n, 2, 2, seed=43)
    out = mx.ffn(layer, x, r, residual)
    _check_ffn(layer, x, r, residual, out)
    assert torch.equal(mx.ffn(layer, x, r, residual), out)
    ws = torch.empty(mx.ffn_workspace_bytes(layer, n), dtype=torch.uint8, device="cuda")
    assert torch.equal(mx.ffn(layer, x, r, residual, ws=ws), out)


@pytest.mark.parametrize("n", [1, 4, 20, 300])
def test_ffn_same_rows_whatever_the_batch(n):
    # a token's result does not depend on the others, nor on the path that its batch takes
    layer = _layer(16, 512, 256, 4, seed=9)
    x, residual = _normal((300, 512), "bf16", seed=3), _normal((300, 512), "f32", seed=4)
    logits = torch.randn((300, 16), generator=_gen(6)).cuda()
    whole = mx.ffn(layer, x, qmoe.route(logits, 4), residual)
    part = mx.ffn(layer, x[:n], qmoe.route(logits[:n], 4), residual[:n].contiguous())
    # the combine's operands are the same fp32 numbers but for their sums' order in two parts
    assert ((whole[:n] - part).abs() <= 4 * 2.0 ** -24 * whole[:n].abs().clamp(min=1.0)).all()


@pytest.mark.parametrize("n", [4, 40])
def test_ffn_repeated_and_missing_experts(n):
    # routing records that no router writes: an expert twice for a token; and, for the window,
    # ids that are no expert, which add nothing
    layer = _layer(6, 128, 64, 4, seed=11)
    x, residual = _normal((n, 128), "bf16", seed=5), _normal((n, 128), "f32", seed=6)
    ids = torch.randint(0, 6, (n, 4), generator=_gen(7), dtype=torch.int32)
    ids[:, 2] = ids[:, 0]
    w = torch.rand((n, 4), generator=_gen(8)).cuda()
    offsets, pairs = mx_ref.grouping(ids.numpy(), 6)
    r = qmoe.Routing(ids.cuda(), w, torch.from_numpy(offsets).cuda(), torch.from_numpy(pairs).cuda())
    _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))
    same = ids * 0 + 3  # all pairs of one expert: more than the 16 of one pass
    offsets, pairs = mx_ref.grouping(same.numpy(), 6)
    r = qmoe.Routing(same.cuda(), w, torch.from_numpy(offsets).cuda(), torch.from_numpy(pairs).cuda())
    _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))
    if n <= 16:
        r.topk_ids[1, 2], r.topk_ids[2, 0] = -1, 6
        _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))


@pytest.mark.parametrize("n", [3, 40, 300])
def test_ffn_pairs_of_no_expert(n):
    # a record that keeps the pairs of some experts only, as a shard of them has it: a token with
    # none of its pairs left keeps its residual, and what the workspace held does not matter
    layer = _layer(6, 128, 64, 4, seed=17)
    x, residual = _normal((n, 128), "bf16", seed=18), _normal((n, 128), "f32", seed=19)
    ids = torch.randint(0, 6, (n, 4), generator=_gen(20), dtype=torch.int32)
    drop = torch.rand((n, 4), generator=_gen(21)) < 0.4
    drop[1] = True
    ids[drop] = torch.where(torch.rand(int(drop.sum()), generator=_gen(22)) < 0.5, -1, 6).int()
    flat = ids.view(-1).numpy()
    pairs = np.argsort(flat, kind="stable")
    pairs = pairs[(flat[pairs] >= 0) & (flat[pairs] < 6)]
    offsets = np.concatenate(([0], np.bincount(flat[pairs], minlength=6).cumsum())).astype(np.int32)
    pairs = np.concatenate((pairs, np.zeros(4 * n - len(pairs)))).astype(np.int32)
    w = torch.rand((n, 4), generator=_gen(23)).cuda()
    r = qmoe.Routing(ids.cuda(), w, torch.from_numpy(offsets).cuda(), torch.from_numpy(pairs).cuda())
    ws = torch.full((mx.ffn_workspace_bytes(layer, n),), 0xff, dtype=torch.uint8, device="cuda")
    out = mx.ffn(layer, x, r, residual, ws=ws)
    _check_ffn(layer, x, r, residual, out)
    assert torch.equal(out[1], residual[1])


@pytest.mark.parametrize("n", [5, 70])
def test_ffn_zero_rows_nan_rows_and_ends(n):
    layer = _layer(8, 256, 128, 2, seed=13)
    x, residual = _normal((n, 256), "f32", seed=7), _normal((n, 256), "f32", seed=8)
    r = _routing(n, 8, 2, seed=9)
    clean = mx.ffn(layer, x, r, residual)
    x[1] = 0
    x[2] *= 2.0 ** -60    # hidden blocks near the least scale
    x[3] *= 2.0 ** 40
    out = mx.ffn(layer, x, r, residual)
    assert torch.equal(out[1], residual[1])
    _check_ffn(layer, x, r, residual, out)
    x[4, 5] = torch.nan
    out2 = mx.ffn(layer, x, r, residual)
    assert out2[4].isnan().all()
    rest = torch.arange(n) != 4
    assert torch.equal(out2[rest.cuda()], out[rest.cuda()]) and torch.equal(out2[0], clean[0])


def test_ffn_hidden_codes_next_to_borders():
    # h just beside a border of the 4-bit grid: with gate so large that silu(g) = g to the last
    # fp32 bit and up = 1, h is g, whose fp32 steps straddle the borders
    d, f, E, k = 64, 32, 1, 1
    for n in (8, 64):
        layer = _layer(E, d, f, k, seed=1)
        x = torch.zeros((n, d))
        x[:, 0] = torch.linspace(1, 6, n)
        x[:, 32] = 1.0
        x = x.cuda()
        r = _routing(n, E, k)
        residual = torch.zeros((n, d)).cuda()
        _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))
    # many values, as they come: no code may differ from the 64-bit one
    layer = _layer(4, 1024, 512, 2, seed=21)
    x = _normal((512, 1024), "bf16", seed=22)
    r = _routing(512, 4, 2, seed=23)
    residual = _normal((512, 1024), "f32", seed=24)
    _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))


@pytest.mark.parametrize("n", [2, 64])
@pytest.mark.parametrize("gate,up,x0", [(-96.0, 2.0 ** 120, 1.0), (2.0 ** -126, 2.0 ** 127, 1.5 * 2.0 ** -22)])
def test_ffn_hidden_of_a_vanishing_gate_and_a_huge_up(n, gate, up, x0):
    # e^-g beyond the fp32 range, or g below its normal numbers, with products in the range
    wg, wu = torch.zeros((32, 64), dtype=torch.float32), torch.zeros((32, 64), dtype=torch.float32)
    wg[:, 0], wu[:, 32] = 1.0, 2.0 ** -10
    wg[5, 0], wu[5, 32] = gate, up
    layer = mx.MxLayer(mx.MxMatrix(*_split(mx.quantize(wg.cuda()), 1)), mx.MxMatrix(*_split(mx.quantize(wu.cuda()), 1)),
                       mx.MxMatrix(*_split(_weights(64, 32, 31), 1)), 1)
    x = torch.zeros((n, 64))
    x[:, 0], x[:, 32] = x0, 1.0
    x, r = x.cuda(), _routing(n, 1, 1)
    residual = torch.zeros((n, 64)).cuda()
    _check_ffn(layer, x, r, residual, mx.ffn(layer, x, r, residual))


def test_ffn_rows_behind_the_last_token():
    layer = _layer(8, 128, 64, 2, seed=15)
    for n in (3, 50):
        x = _normal((n, 160), "bf16", seed=n)[:, :128]  # rows further apart than they are long
        r = _routing(n, 8, 2)
        frame = torch.full((n + 4, 128), 3.0).cuda()
        residual = frame[:n]
        ref = mx.ffn(layer, x.contiguous(), r, residual)
        mx.ffn(layer, x, r, residual, out=residual)
        assert torch.equal(frame[:n], ref) and (frame[n:] == 3.0).all()
    assert mx.ffn(layer, _normal((0, 128)), qmoe.Routing.empty(0, 8, 2)).shape == (0, 128)


# ---------------------------------------------------------------- as they are used


def test_a_layer_router_projection_experts():
    """One decoder layer's second half: router logits and a projection from one quantization,
    routing by a rule in groups, experts into the residual; prompt and then single tokens."""
    E, d, f, k = 32, 512, 256, 4
    layer = _layer(E, d, f, k, seed=31)
    router, proj = _weights(E, d, seed=34), _weights(d, d, seed=35)
    rule = qmoe.RouteRule(bias=_normal((E,), "f32", 36, 0.1), groups=8, top_groups=4, scale=2.0)

    def half(x, residual):
        q = mx.quantize(x)
        r = qmoe.route_scored(mx.linear(q, router, dtype=torch.float32), k, rule)
        y = mx.linear(q, proj, dtype=torch.float32)
        return mx.ffn(layer, x, r, residual + y), r

    x, residual = _normal((90, d), "bf16", 37), _normal((90, d), "f32", 38)
    whole, r = half(x, residual)
    q = mx_ref.rounded(x)
    logits = (q @ mx_ref.matrix(router).T).float()
    ids, w = mx_ref.route(logits.cpu().numpy(), k, "sigmoid", rule.bias.cpu().numpy(), 8, 4, True, True, 2.0)
    assert np.array_equal(r.topk_ids.cpu().numpy(), ids)
    start = residual + (q @ mx_ref.matrix(proj).T).float()
    ref, bound = mx_ref.ffn(layer, x, torch.from_numpy(ids).long().cuda(),
                            torch.from_numpy(w).float().cuda(), start)
    assert ((whole.double() - ref).abs() <= bound + ref.abs() * 2.0 ** -22).all()
    for t in (0, 41, 89):
        one, _ = half(x[t: t + 1], residual[t: t + 1])
        assert ((one[0] - whole[t]).abs() <= 4 * 2.0 ** -24 * whole[t].abs().clamp(min=1.0)).all()


def test_routing_by_a_rule_feeds_the_block_quantized_layer():
    from quantized_routed_expert_router_amd import synth, workloads
    w = synth.config(1)
    layer = workloads.device_layer(w, 0)
    lg, x = synth.layer_inputs(w, 0)
    logits, xd = torch.from_numpy(lg).cuda(), torch.from_numpy(x).cuda()
    a, b = xd.clone(), xd.clone()
    qmoe.ffn_decode(layer, xd, qmoe.route(logits, w.k), a)
    qmoe.ffn_decode(layer, xd, qmoe.route_scored(logits, w.k, qmoe.RouteRule(score="softmax")), b)
    assert torch.allclose(a, b, rtol=0, atol=2.0 ** -20)


@pytest.mark.parametrize("n", [1, 12, 150])
def test_captured_replayed_and_beside_another_graph(n):
    E, d, f, k = 16, 256, 128, 4
    layer, proj = _layer(E, d, f, k, seed=41), _weights(d, d, seed=44)
    rule = qmoe.RouteRule(groups=4, top_groups=2)
    state = []
    for i in range(2):
        s = dict(x=_normal((n, d), "bf16", 45 + i), res=_normal((n, d), "f32", 47 + i), logits=_normal((n, E), "f32", 49 + i))
        s["ws"] = torch.empty(max(mx.ffn_workspace_bytes(layer, n), 256), dtype=torch.uint8, device="cuda")
        s["r"], s["rws"] = qmoe.Routing.empty(n, E, k), qmoe.route_workspace(n, E, k)
        s["out"], s["y"] = torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda", dtype=torch.bfloat16)
        state.append(s)

    def step(s):
        qmoe.route_scored(s["logits"], k, rule, out=s["r"], ws=s["rws"])
        mx.ffn(layer, s["x"], s["r"], s["res"], out=s["out"], ws=s["ws"])
        mx.linear(s["x"], proj, out=s["y"])
        return mx.dequantize(mx.quantize(s["x"]))

    graphs = []
    for s in state:
        step(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s["deq"] = step(s)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for i, s in enumerate(state):
            s["x"].copy_(_normal((n, d), "bf16", 60 + 2 * turn + i))
            s["logits"].copy_(_normal((n, E), "f32", 70 + 2 * turn + i))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):  # both at once
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s in state:
            r = qmoe.route_scored(s["logits"], k, rule)
            assert torch.equal(s["out"], mx.ffn(layer, s["x"], r, s["res"]))
            assert torch.equal(s["y"], mx.linear(s["x"], proj))
            assert torch.equal(s["deq"], mx.dequantize(mx.quantize(s["x"])))


def test_another_stream():
    layer, w = _layer(8, 256, 128, 2, seed=51), _weights(300, 256, seed=52)
    side = torch.cuda.Stream()
    for n in (2, 80):
        x, residual = _normal((n, 256), "bf16", n), _normal((n, 256), "f32", n + 1)
        r = _routing(n, 8, 2)
        side.wait_stream(torch.cuda.current_stream())
        a = [mx.linear(x, w, stream=side), mx.ffn(layer, x, r, residual, stream=side),
             mx.dequantize(mx.quantize(x, stream=side), stream=side)]
        side.synchronize()
        b = [mx.linear(x, w), mx.ffn(layer, x, r, residual), mx.dequantize(mx.quantize(x))]
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_refusals():
    x = _normal((4, 64))
    w = _weights(8, 64, seed=1)
    layer, r = _layer(4, 64, 32, 2), _routing(4, 4, 2)
    bad_w = mx.MxMatrix(w.codes, w.scales[:, :1].contiguous())
    for call in (lambda: mx.quantize(x[:, :40]), lambda: mx.quantize(x.t()), lambda: mx.quantize(x.double()),
                 lambda: mx.quantize(x.cpu()), lambda: mx.quantize(x[0]), lambda: mx.quantize(x, out=w),
                 lambda: mx.linear(x[:, :32], w), lambda: mx.linear(x, bad_w), lambda: mx.linear(x.cpu(), w),
                 lambda: mx.linear(x, w, dtype=torch.float64), lambda: mx.linear(x, w, out=torch.empty((4, 9)).cuda()),
                 lambda: mx.linear(x, mx.MxMatrix(w.codes.cpu(), w.scales.cpu())),
                 lambda: mx.linear(x, mx.MxMatrix(w.codes.int(), w.scales)),
                 lambda: mx.dequantize(w, torch.int32), lambda: mx.dequantize(bad_w),
                 lambda: mx.ffn(layer, x[:, :32], r), lambda: mx.ffn(layer, x, r, x),
                 lambda: mx.ffn(layer, x, r, torch.zeros((3, 64)).cuda()),
                 lambda: mx.ffn(mx.MxLayer(layer.gate, layer.down, layer.up, 2), x, r),
                 lambda: mx.ffn(layer, x, r, torch.zeros((4, 64)).cuda(), out=torch.zeros((4, 32)).cuda())):
        with pytest.raises(ValueError):
            call()
    res = torch.zeros((4, 64)).cuda()
    both = torch.zeros((8, 64)).cuda()
    odd = torch.zeros(4 * 64 + 1).cuda()[1:].view(4, 64)
    for call in (lambda: mx.ffn(mx.MxLayer(layer.gate, layer.up, layer.down, 5), x, qmoe.Routing.empty(8, 4, 5)),
                 lambda: mx.ffn(layer, x, r, both[1:5], out=both[2:6]), lambda: mx.ffn(layer, x, r, odd),
                 lambda: mx.ffn(layer, x, r, res, out=odd),
                 lambda: mx.linear(_normal((4, 65))[:, 1:], w),
                 lambda: mx.linear(_normal((4, 66))[:, :64], w),
                 lambda: mx.ffn(layer, x, r, res, ws=torch.empty(256, dtype=torch.uint8).cuda()[:8]),
                 lambda: mx.quantize(_normal((40, 64)).view(-1)[4: 4 + 1280].view(20, 64))):
        with pytest.raises(qmoe.MoeError):
            call()
