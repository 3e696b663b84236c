"""Microscaled 4-bit floats and routing by a rule, from their definitions in 64 bits, in plain
numpy and torch; shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x: np.ndarray):
    """(codes [..., K], scale bytes [..., K / 32]) of float64 rows."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    _, e = np.frexp(np.where(bad, 1.0, top))
    e = np.where(top == 0, -127, np.clip(e - 3, -127, 127))
    y = np.where(bad[..., None], 0.0, b) * np.exp2(-e.astype(np.float64))[..., None]
    # nearest grid value, ties to the even code
    d = np.abs(np.abs(y)[..., None] - GRID)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(np.abs(y) >= 6, 7, code) | (np.signbit(y) * 8)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return code[..., 0::2] | code[..., 1::2] << 4


def values(packed, scales) -> np.ndarray:
    """float64 values of packed codes and scale bytes (255: NaN)."""
    packed, scales = np.asarray(packed), np.asarray(scales)
    code = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, -1)


def matrix(m) -> torch.Tensor:
    """float64 values of a library matrix, on its device."""
    return torch.from_numpy(values(m.codes.cpu().numpy(), m.scales.cpu().numpy())).to(m.codes.device)


def rounded(x: torch.Tensor) -> torch.Tensor:
    """Q(x) in float64."""
    code, scale = quantize(x.double().cpu().numpy())
    return torch.from_numpy(values(pack(code), scale)).to(x.device)


def silu_up(g: torch.Tensor, u: torch.Tensor) -> torch.Tensor:
    return g / (1 + torch.exp(-g)) * u


def ffn(layer, x, ids, weights, residual):
    """(out, largest possible rounding) in float64; expert by expert."""
    q, n, k = rounded(x), x.shape[0], ids.shape[1]
    out = residual.double().clone()
    size = residual.double().abs()
    gate, up, down = (matrix(m) for m in (layer.gate, layer.up, layer.down))
    for e in range(gate.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        g, u = q[t] @ gate[e].T, q[t] @ up[e].T
        # the library's sums are exact where these are fp32 numbers of few enough bits
        assert torch.equal(g.float().double(), g) and torch.equal(u.float().double(), u)
        y = rounded(silu_up(g, u)) @ down[e].T
        w = weights[t, j].double()[:, None]
        out.index_add_(0, t, w * y)
        size.index_add_(0, t, (w * y).abs())
    # y rounded to fp32 in sums of exact products (a few partial sums), then the output
    return out, size * (8 * 2.0 ** -24)


def route(logits: np.ndarray, k: int, score: str, bias, groups: int, keep: int, top2: bool,
          renormalize: bool, scale: float):
    """ids and weights of each token, a token at a time."""
    n, E = logits.shape
    ids, w = np.zeros((n, k), np.int32), np.zeros((n, k))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(n):
        l = logits[t].astype(np.float64)
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-l))
            else:
                m = np.nanmax(np.where(np.isnan(l), -np.inf, l))
                p = np.where(l == m, 1.0, np.exp(l - m))
                p = np.where(np.isnan(l) | (l == -np.inf), 0.0, p)
                s = p / p.sum() if p.sum() > 0 else np.zeros(E)
            c = s + b
        last = np.isnan(l) | np.isnan(c) | (c == -np.inf)
        c = np.where(last, -np.inf, c)
        s = np.where(last | (l == -np.inf), 0.0, s)
        by = c.reshape(groups, -1)
        inside = -np.sort(-by, -1)
        worth = inside[:, :2].sum(-1) if top2 and by.shape[1] > 1 else inside[:, 0]
        worth = np.where(np.isnan(worth), -np.inf, worth)
        stay = np.argsort(-worth, kind="stable")[:keep]
        where = np.sort(np.concatenate([np.arange(g * by.shape[1], (g + 1) * by.shape[1]) for g in stay]))
        ids[t] = where[np.argsort(-c[where], kind="stable")[:k]]
        v = s[ids[t]]
        if renormalize:
            v = v / v.sum() if v.sum() > 0 else np.zeros(k)
        w[t] = v * scale
    return ids, w


def grouping(ids: np.ndarray, E: int):
    flat = ids.ravel()
    offsets = np.concatenate(([0], np.bincount(flat, minlength=E).cumsum())).astype(np.int32)
    return offsets, np.argsort(flat, kind="stable").astype(np.int32)
