"""The 4-bit form of the hidden vector against that of its binary64 value, for the window (up to
16 tokens) and for the grouped products."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mx_ref
from quantized_routed_expert_router_amd import mx, qmoe

pytestmark = pytest.mark.gpu

TOKENS = [3, 16, 17, 64, 200]


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _quantized(shape, seed):
    return mx.quantize((torch.randn(shape, generator=_gen(seed)) * 0.02).cuda())


def _to(experts, E):
    """The routing record of one expert a token, with weight 1."""
    ids = torch.as_tensor(experts, dtype=torch.int32).view(-1, 1)
    offsets, pairs = mx_ref.grouping(ids.numpy(), E)
    return qmoe.Routing(ids.cuda(), torch.ones((len(ids), 1)).cuda(), torch.from_numpy(offsets).cuda(),
                        torch.from_numpy(pairs).cuda())


@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("d", [96, 256])
def test_nan_beside_zeros(n, which, d):
    """A row of zeros under a NaN scale of gate, or of up, alone: that sum is NaN, the other 0 and
    every other value of the block 0. The block is NaN, and with it the token's outputs."""
    E, f = 2, 64
    layer = mx.MxLayer(_quantized((E, f, d), 1), _quantized((E, f, d), 2), _quantized((E, d, f), 3), 1)
    getattr(layer, which).scales[0, 37, 1] = 255
    x = torch.randn((n, d), generator=_gen(4)).cuda()
    x[::2] = 0
    x[1] = 0
    experts = torch.arange(n) % 2  # expert 0 has rows of zeros alone, expert 1 has one
    out = mx.ffn(layer, x, _to(experts, E), torch.zeros((n, d)).cuda())
    assert out[::2].isnan().all()
    assert torch.isfinite(out[1::2]).all() and (out[1] == 0).all()


@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("zero", ["gate", "up"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinity_beside_zeros(n, zero, sign):
    """One factor's sum beyond fp32, the other's 0: their product is NaN in binary64 too."""
    d, f = 64, 32
    w = torch.zeros((f, d))
    big = torch.zeros((f, d))
    big[7, 0] = sign * 2.0 ** 127
    big, w = mx.quantize(big.cuda()), mx.quantize(w.cuda())
    x = torch.zeros((n, d)).cuda()
    x[:, 0] = 2.0 ** 20
    x[1] = 0  # 0 times 0
    sums = mx.linear(x, big, dtype=torch.float32)
    assert not sums[0, 7].isfinite() and (sums[1] == 0).all()
    pair = (w, big) if zero == "gate" else (big, w)
    layer = mx.MxLayer(*(mx.MxMatrix(m.codes[None], m.scales[None]) for m in pair), _quantized((1, d, f), 5), 1)
    residual = torch.ones((n, d)).cuda()
    out = mx.ffn(layer, x, _to([0] * n, 1), residual)
    assert out[0].isnan().all() and out[2:].isnan().all() and torch.equal(out[1], residual[1])


# ---------------------------------------------------------------- next to the borders


def _exactly(values, blocks):
    """A matrix [rows, 32 blocks] whose rows, multiplied with a row that is 1 at the first column of
    each block, sum to the fp32 `values`: two bits of the significand a block."""
    v = np.asarray(values, np.float64).ravel()
    m, e = np.frexp(np.abs(v))
    whole = np.rint(m * 2.0 ** 24).astype(np.int64)
    assert (whole * np.exp2(e - 24.0) == np.abs(v)).all()
    codes = np.zeros((len(v), 32 * blocks), np.uint8)
    scales = np.zeros((len(v), blocks), np.uint8)
    for b in range(12):
        piece = whole >> (22 - 2 * b) & 3
        codes[:, 32 * b] = np.array([0, 2, 4, 5])[piece] | np.where(v < 0, 8, 0)
        scales[:, b] = 127 + e - 2 - 2 * b
    return mx.MxMatrix(torch.from_numpy(mx_ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda())


def _near_borders(shape, seed):
    """fp32 gate and up sums whose h lies within a few 2^-23 of itself of a border between two codes
    and, for the largest of every second block, of a border between two scales."""
    rng = np.random.default_rng(seed)
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    h = borders[rng.integers(0, 7, (*shape, 32))]
    top = np.where(np.arange(shape[-1]) % 2 == 0, 4.0, 5.0)
    h[..., 5] = top
    h[:, ::2][h[:, ::2] > 4.0] = 3.5  # the largest is the one on the scale's border
    h *= np.exp2(rng.integers(-6, 7, (*shape, 1)))
    g = (rng.normal(size=h.shape) * 4).astype(np.float32)
    g = np.where(np.abs(g) < 2.0 ** -6, np.float32(1.5), g).astype(np.float64)
    sign = rng.choice([-1.0, 1.0], h.shape)
    u = (sign * h / (g / (1 + np.exp(-g)))).astype(np.float32)
    for _ in range(3):
        u = np.nextafter(u, (u * rng.choice([0.5, 1.0, 2.0], u.shape)).astype(np.float32))
    return g.reshape(shape[0], -1), u.astype(np.float64).reshape(shape[0], -1)


@pytest.mark.parametrize("d", [384, 512])
@pytest.mark.parametrize("form", ["window", "grouped", "many"])
def test_codes_next_to_borders(d, form):
    """The down matrix is the identity and the weights are 1: the output is Q(h) itself."""
    E, blocks = 24, d // 32
    g, u = _near_borders((E, blocks), d)
    gate, up = _exactly(g, blocks), _exactly(u, blocks)
    eye = mx.quantize(torch.eye(d).cuda())
    shaped = lambda m: mx.MxMatrix(m.codes.view(E, d, -1), m.scales.view(E, d, -1))  # noqa: E731
    layer = mx.MxLayer(shaped(gate), shaped(up), mx.MxMatrix(eye.codes.repeat(E, 1, 1), eye.scales.repeat(E, 1, 1)), 1)
    ones = torch.zeros((64, d)).cuda()
    ones[:, ::32] = 1.0
    for rows in (1, 64):  # the sums are the wanted numbers to the last bit
        for m, want in ((gate, g), (up, u)):
            got = mx.linear(ones[:rows], m, dtype=torch.float32)
            assert np.array_equal(got.cpu().double().numpy(), np.broadcast_to(want.ravel(), got.shape))
    h = g / (1 + np.exp(-g)) * u
    code, scale = mx_ref.quantize(h)
    q = mx_ref.values(mx_ref.pack(code), scale)
    # these values do straddle the borders: nudged by 2^-21 either way most get another code or scale
    lo, hi = (np.stack(np.broadcast_arrays(*(a.reshape(E, blocks, -1) for a in mx_ref.quantize(h * s))), -1)
              for s in (1 - 2.0 ** -21, 1 + 2.0 ** -21))
    assert (lo != hi).any(-1).mean() > 0.5
    if form == "window":
        calls = [list(range(i, i + 8)) for i in range(0, E, 8)]
    elif form == "grouped":
        calls = [[i % E for i in range(2 * E)]]
    else:  # tiles of up to 128, 64 and 32 pairs
        calls = [[0] * 100 + [1] * 50 + list(range(E))]
    for experts in calls:
        out = mx.ffn(layer, ones[:1].repeat(len(experts), 1), _to(experts, E))
        assert np.array_equal(out.cpu().double().numpy(), q[experts])
