"""Rows and outputs of the dense microscaled product side by side in one buffer, and scales that
end where other memory begins."""
from __future__ import annotations

import pytest
import torch

from quantized_routed_expert_router_amd import mx, qmoe

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _quantized(shape, seed):
    return mx.quantize((torch.randn(shape, generator=_gen(seed)) * 0.02).cuda())


@pytest.mark.parametrize("n", [1, 2, 16, 40, 700])
@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("first", ["x", "out"])
def test_rows_and_outputs_in_one_frame(n, kinds, first):
    K, N = 160, 72
    w = _quantized((N, K), 3)
    dx, do = (TYPES[k] for k in kinds)
    bx, bo = K * dx.itemsize, N * do.itemsize
    frame = torch.full((n, bx + bo + 32), 0x55, dtype=torch.uint8).cuda()
    ax, ao = (0, bx) if first == "x" else (bo + 16, 16)
    if first == "x":
        ao += 16
    x, out = frame[:, ax: ax + bx].view(dx), frame[:, ao: ao + bo].view(do)
    rows = torch.randn((n, K), generator=_gen(n)).to(dx)
    x.copy_(rows)
    ref = mx.linear(rows.cuda(), w, dtype=do)
    assert mx.linear(x, w, out=out) is out and torch.equal(out, ref)
    assert torch.equal(x.cpu(), rows)
    out.zero_()
    x.zero_()
    used = torch.zeros(frame.shape[1], dtype=torch.bool)
    used[ax: ax + bx] = used[ao: ao + bo] = True
    assert (frame[:, ~used.cuda()] == 0x55).all()


def _between(t, before=64, after=64):
    """The bytes of `t` in memory between NaN scales."""
    arena = torch.full((before + t.numel() + after,), 255, dtype=torch.uint8).cuda()
    view = arena[before: before + t.numel()]
    view.copy_(t.view(-1))
    return view.view(t.shape)


@pytest.mark.parametrize("n,K,N", [(3, 32, 16), (20, 32, 16), (33, 32, 17), (33, 64, 9), (64, 96, 19), (40, 288, 21),
                                   (70, 544, 65), (300, 416, 1001)])
def test_scales_between_other_bytes(n, K, N):
    # rows of scales are read in whole requests: what lies before and behind them does not matter
    w, x = _quantized((N, K), N), torch.randn((n, K), generator=_gen(n)).bfloat16().cuda()
    q = mx.quantize(x)
    ref = mx.linear(q, w, dtype=torch.float32)
    placed = mx.MxMatrix(w.codes, _between(w.scales))
    assert torch.isfinite(ref).all()
    assert torch.equal(mx.linear(q, placed, dtype=torch.float32), ref)
    assert torch.equal(mx.linear(mx.MxMatrix(q.codes, _between(q.scales)), placed, dtype=torch.float32), ref)


@pytest.mark.parametrize("n", [3, 40, 300])
@pytest.mark.parametrize("d,f", [(32, 32), (96, 32), (160, 96), (256, 288)])
def test_scales_of_experts_between_other_bytes(n, d, f):
    E, k = 5, 2
    gate, up, down = _quantized((E, f, d), 1), _quantized((E, f, d), 2), _quantized((E, d, f), 3)
    x, residual = torch.randn((n, d), generator=_gen(n)).cuda(), torch.randn((n, d), generator=_gen(4)).cuda()
    r = qmoe.route(torch.randn((n, E), generator=_gen(5)).cuda(), k)
    ref = mx.ffn(mx.MxLayer(gate, up, down, k), x, r, residual)
    layer = mx.MxLayer(*(mx.MxMatrix(m.codes, _between(m.scales)) for m in (gate, up, down)), k)
    assert torch.isfinite(ref).all()
    assert torch.equal(mx.ffn(layer, x, r, residual), ref)
