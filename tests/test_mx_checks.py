"""Routing by a rule and the microscaled products without a GPU: argument checks of the C ABI
(every call here is refused, or has nothing to do), workspace sizes, and the binding's checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

from quantized_routed_expert_router_amd import mx, qmoe

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 0x7f0000000000  # aligned addresses that are never dereferenced here
lib, ref = qmoe.lib, ctypes.byref
BF16, F16, E4M3, F32 = 0, 1, 2, 3


def at(i: int) -> int:
    return FAKE + (i << 32)


def _rule(score=0, bias=None, groups=1, top_groups=1, group_score=0, renormalize=1, scale=1.0):
    return qmoe._RouteRule(score, bias, groups, top_groups, group_score, renormalize, scale)


def _route(rule, n=4, E=32, k=4, dtype=F32, logits=at(1), out=None, ws=at(9), ws_bytes=1 << 30):
    out = out or qmoe._Routing(at(2), at(3), at(4), at(5))
    return lib.moe_route_scored(logits, dtype, n, E, k, ref(rule) if rule else None, ref(out), ws, ws_bytes, None)


def test_route_rule_refusals():
    for kw in (dict(n=-1), dict(n=65537), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=1024, k=65),
               dict(logits=None), dict(logits=at(1) + 2), dict(out=qmoe._Routing(None, at(3), at(4), at(5))),
               dict(out=qmoe._Routing(at(2), None, at(4), at(5))), dict(out=qmoe._Routing(at(2), at(3), None, at(5))),
               dict(out=qmoe._Routing(at(2), at(3), at(4), None)), dict(out=qmoe._Routing(at(1), at(3), at(4), at(5)))):
        assert _route(_rule(), **kw) == INVALID, kw
    assert _route(None) == INVALID
    for dtype in (E4M3, -1, 4):
        assert _route(_rule(), dtype=dtype) == UNSUPPORTED
    for kw in (dict(score=2), dict(score=-1), dict(group_score=2), dict(groups=0), dict(groups=5), dict(groups=64),
               dict(groups=8, top_groups=0), dict(groups=8, top_groups=9), dict(groups=16, top_groups=1),
               dict(renormalize=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(bias=at(7) + 1),
               dict(bias=at(3))):
        assert _route(_rule(**kw)) == INVALID, kw
    assert _route(_rule(groups=65, top_groups=65), E=65, k=1) == INVALID  # more groups than the limit
    need = lib.moe_route_workspace_bytes(65536, 32, 4)
    assert _route(_rule(), n=65536, ws=None) == WS_SMALL and _route(_rule(), n=65536, ws_bytes=need - 1) == WS_SMALL
    assert _route(_rule(), n=65536, ws=at(9) + 128) == INVALID


def test_route_outputs_that_overlap_are_refused():
    # 4 tokens of 4 experts each: 64 bytes an output; 65536 tokens of 32 experts also use ws
    for kw in (dict(out=qmoe._Routing(at(2), at(2) + 60, at(4), at(5))), dict(out=qmoe._Routing(at(2), at(3), at(2), at(5))),
               dict(out=qmoe._Routing(at(2), at(3), at(4), at(4) + 60)), dict(out=qmoe._Routing(at(2) + 2, at(3), at(4), at(5))),
               dict(out=qmoe._Routing(at(2), at(3), at(4), at(5) + 1)), dict(n=0, out=qmoe._Routing(None, None, None, at(5) + 2)),
               dict(n=65536, ws=at(1)), dict(n=65536, ws=at(2)), dict(n=65536, ws=at(5))):
        assert _route(_rule(), **kw) == INVALID, kw
    assert _route(_rule(bias=at(9) + 256), n=65536) == INVALID


def test_quantize_refusals():
    q = lib.moe_mx_quantize
    assert q(at(1), BF16, 0, 64, 64, None, None, None) == OK
    assert q(None, BF16, 0, 64, 64, None, None, None) == OK
    for args in ((None, BF16, 4, 64, 64, at(2), at(3)), (at(1) + 8, BF16, 4, 64, 64, at(2), at(3)),
                 (at(1), BF16, -1, 64, 64, at(2), at(3)), (at(1), BF16, 4, 48, 48, at(2), at(3)),
                 (at(1), BF16, 4, 0, 64, at(2), at(3)), (at(1), BF16, 4, 65568, 65568, at(2), at(3)),
                 (at(1), BF16, 4, 64, 68, at(2), at(3)), (at(1), BF16, 4, 64, -64, at(2), at(3)),
                 (at(1), BF16, 4, 64, 64, None, at(3)), (at(1), BF16, 4, 64, 64, at(2), None),
                 (at(1), BF16, 4, 64, 64, at(2) + 8, at(3)), (at(1), BF16, 4, 64, 64, at(2), at(3) + 4),
                 (at(1), BF16, 4, 64, 64, at(1) + 496, at(3)), (at(1), BF16, 4, 64, 64, at(2), at(1)),
                 (at(1), BF16, 4, 64, 64, at(2), at(2) + 112), (at(1), BF16, 1 << 62, 64, 64, at(2), at(3))):
        assert q(*args, None) == INVALID, args
    for dtype in (E4M3, 7):
        assert q(at(1), dtype, 4, 64, 64, at(2), at(3), None) == UNSUPPORTED


def _mat(rows=8, cols=64, codes=at(2), scales=at(3)):
    return mx._MxMatrix(codes, scales, rows, cols)


def test_dequantize_refusals():
    d = lib.moe_mx_dequantize
    assert d(ref(_mat()), 0, F32, None, None) == OK
    assert d(None, 4, F32, at(1), None) == INVALID
    assert d(ref(_mat()), 4, E4M3, at(1), None) == UNSUPPORTED
    for m, rows, out in ((_mat(cols=40), 4, at(1)), (_mat(codes=None), 4, at(1)), (_mat(scales=None), 4, at(1)),
                         (_mat(codes=at(2) + 4), 4, at(1)), (_mat(), -1, at(1)), (_mat(), 4, None),
                         (_mat(), 4, at(1) + 4), (_mat(), 4, at(2) + 64), (_mat(), 4, at(3)), (_mat(), 1 << 62, at(1))):
        assert d(ref(m), rows, F32, out, None) == INVALID


def _linear(w, n=4, x=at(1), dtype=BF16, stride=64, out=at(4), out_dtype=F32, out_stride=8, ws=None, ws_bytes=0):
    return lib.moe_mx_linear(x, dtype, stride, n, ref(w) if w else None, out, out_dtype, out_stride, ws, ws_bytes, None)


def test_linear_refusals():
    assert _linear(_mat(), n=0, x=None, out=None) == OK
    assert _linear(_mat(), n=0, out_dtype=E4M3) == UNSUPPORTED
    assert _linear(None) == INVALID
    for kw in (dict(n=-1), dict(n=65537), dict(x=None), dict(x=at(1) + 4), dict(stride=60), dict(stride=-64),
               dict(out=None), dict(out=at(4) + 2), dict(out_stride=7), dict(out=at(1) + 256), dict(out=at(2)),
               dict(out=at(3)), dict(out_stride=1 << 60)):
        assert _linear(_mat(), **kw) == INVALID, kw
    for w in (_mat(rows=0), _mat(rows=(1 << 24) + 1), _mat(cols=33), _mat(cols=0), _mat(cols=65568),
              _mat(codes=None), _mat(scales=None), _mat(codes=at(2) + 8), _mat(scales=at(3) + 8)):
        assert _linear(w) == INVALID
    assert _linear(_mat(), dtype=E4M3) == UNSUPPORTED and _linear(_mat(), out_dtype=E4M3) == UNSUPPORTED
    need = lib.moe_mx_linear_workspace_bytes(40, 64)
    assert need >= 40 * 34
    assert _linear(_mat(), n=40) == WS_SMALL
    assert _linear(_mat(), n=40, ws=at(8), ws_bytes=need - 1) == WS_SMALL
    for ws in (at(8) + 16, at(4), at(1), at(2), at(3)):
        assert _linear(_mat(), n=40, ws=ws, ws_bytes=1 << 20) == INVALID
    q = lib.moe_mx_linear_quantized
    x = _mat(rows=4, codes=at(5), scales=at(6))
    assert q(ref(_mat(rows=0, codes=None)), ref(_mat()), None, F32, 8, None) == OK
    assert q(None, ref(_mat()), at(4), F32, 8, None) == INVALID
    assert q(ref(x), None, at(4), F32, 8, None) == INVALID
    assert q(ref(_mat(rows=4, cols=96)), ref(_mat()), at(4), F32, 8, None) == INVALID
    for out in (at(5), at(6), at(2), at(3), None):
        assert q(ref(x), ref(_mat()), out, F32, 8, None) == INVALID


def test_linear_workspace_sizes():
    size = lib.moe_mx_linear_workspace_bytes
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 33) == 0 and size(65537, 64) == 0 and size(4, 65568) == 0
    for n in (17, 100, 65536):
        for cols in (32, 2080, 65536):
            assert size(n, cols) >= n * cols // 2 + n * cols // 32 and size(n, cols) % 256 == 0


def _layer(d=64, f=32, E=4, k=2, gate=None, up=None, down=None):
    return mx._MxLayer(d, f, E, k, gate or _mat(f, d, at(10), at(11)), up or _mat(f, d, at(12), at(13)),
                       down or _mat(d, f, at(14), at(15)))


def _ffn(L, n=4, x=at(1), dtype=BF16, stride=64, r=None, residual=at(6), out=at(7), ws=at(8), ws_bytes=1 << 40):
    r = r or qmoe._Routing(at(2), at(3), at(4), at(5))
    return lib.moe_mx_ffn(ref(L) if L else None, x, dtype, stride, n, ref(r), residual, out, ws, ws_bytes, None)


def test_ffn_refusals():
    assert _ffn(_layer(), n=0, x=None, out=None, ws=None, ws_bytes=0) == OK
    assert _ffn(None) == INVALID
    for L in (_layer(d=0), _layer(d=48), _layer(d=8224), _layer(f=0), _layer(f=40), _layer(f=8224), _layer(E=0),
              _layer(E=1025), _layer(k=0), _layer(k=5), _layer(E=128, k=65), _layer(gate=_mat(32, 32)),
              _layer(up=_mat(64, 64)), _layer(down=_mat(32, 64)), _layer(gate=_mat(32, 64, None)),
              _layer(up=_mat(32, 64, at(2), at(3) + 4)), _layer(down=_mat(64, 32, at(2) + 8))):
        assert _ffn(L) == INVALID
    for kw in (dict(n=-1), dict(n=8193), dict(x=None), dict(x=at(1) + 2), dict(stride=68), dict(out=None),
               dict(out=at(7) + 4), dict(residual=at(6) + 4), dict(residual=at(7) + 16), dict(out=at(1) + 480),
               dict(out=at(10)), dict(out=at(15)), dict(out=at(2)), dict(out=at(5)), dict(ws=at(8) + 16),
               dict(ws=at(7)), dict(ws=at(6)), dict(ws=at(14)), dict(ws=at(3)),
               dict(r=qmoe._Routing(None, at(3), at(4), at(5))), dict(r=qmoe._Routing(at(2), at(3), at(4), None))):
        assert _ffn(_layer(), **kw) == INVALID, kw
    assert _ffn(_layer(), dtype=E4M3) == UNSUPPORTED
    need = lib.moe_mx_ffn_workspace_bytes(ref(_layer()), 4)
    assert need > 0 and _ffn(_layer(), ws=None) == WS_SMALL and _ffn(_layer(), ws_bytes=need - 1) == WS_SMALL


def test_ffn_workspace_sizes():
    size = lib.moe_mx_ffn_workspace_bytes
    assert size(None, 4) == 0 and size(ref(_layer(d=48)), 4) == 0 and size(ref(_layer()), 8193) == 0
    assert size(ref(_layer()), 0) == 0
    for n in (1, 16, 17, 500, 8192):
        for d, f, E, k in ((64, 32, 4, 2), (2048, 768, 512, 10), (8192, 8192, 1024, 64)):
            got = size(ref(_layer(d, f, E, k)), n)
            assert got % 256 == 0 and got >= n * k * (f // 2 + f // 32)
    with pytest.raises(ValueError):
        mx.ffn_workspace_bytes(mx.MxLayer(*[mx.MxMatrix(torch.zeros(2, 3), torch.zeros(2, 3))] * 3, 1), 4)


def test_binding_refuses_cpu_tensors_and_shapes():
    u8 = torch.uint8
    w = mx.MxMatrix(torch.zeros((8, 32), dtype=u8), torch.zeros((8, 2), dtype=u8))
    x = torch.zeros((4, 64))
    for call in (lambda: mx.quantize(x), lambda: mx.dequantize(w), lambda: mx.linear(x, w), lambda: mx.linear(w, w),
                 lambda: mx.quantize(torch.zeros((4, 40))), lambda: mx.quantize([1.0]), lambda: mx.linear(None, w),
                 lambda: mx.MxMatrix.empty(4, 40), lambda: mx.MxMatrix.empty(64),
                 lambda: qmoe.route_scored(x, 2, qmoe.RouteRule()), lambda: qmoe.route_scored(x[0], 2, qmoe.RouteRule())):
        with pytest.raises(ValueError):
            call()
    m = mx.MxMatrix.empty(3, 5, 96, device="cpu")
    assert (m.rows, m.cols) == (5, 96) and m.codes.shape == (3, 5, 48) and m.scales.shape == (3, 5, 3)


def test_binding_refuses_more_rows_than_fit_an_int():
    w = mx.MxMatrix(torch.zeros((8, 16), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.uint8))
    with pytest.raises(ValueError, match="rows"):
        mx.linear(torch.zeros((1, 32)).expand(2 ** 32 + 4, 32), w)


def test_launch_splits():
    """The work list's shares: every tile is in one XCD's run, and no run is longer than the grid
    that the host launches for it (the arithmetic of the tile kernel, in Python)."""
    import random
    rng = random.Random(1)
    cost_w, bm = 4, 128
    for _ in range(300):
        E = rng.choice([1, 3, 64, 512, 1024])
        m = [rng.choice([0, 0, 1, rng.randint(0, 40), rng.randint(0, 3000)]) for _ in range(E)]
        tiles = [min(bm, v - i) for v in m for i in range(0, v, bm)]
        costs = [cost_w + -(-r // 32) for r in tiles]
        total, before, first = sum(costs), 0, {8: len(tiles)}
        for j, c in enumerate(costs):
            for x in range(8):
                if x * total == before * 8:
                    first[x] = j
                elif before * 8 < x * total < (before + c) * 8:
                    first[x] = j + 1
            before += c
        if not tiles:
            continue
        assert sorted(first) == list(range(9)) and all(first[x] <= first[x + 1] for x in range(8))
        P = sum(m)
        most = (P + min(E, P) * (bm - 1)) // bm  # the host's bound of the number of tiles
        assert most >= len(tiles)
        limit = min(most, (cost_w + 4) * (-(-most // 8) + 1) // (cost_w + 1) + 2)
        assert max(first[x + 1] - first[x] for x in range(8)) <= limit
