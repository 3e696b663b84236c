"""Plain 64-bit forms of the attention-half operators, on the CPU, and the error bounds
that their tests use. Independent of the library: everything is written from the formulas
of include/qmoe.h."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}
# spacing of the subnormals, halved
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}


def norm_rope(x, weight, positions, inv_freq, eps, offset=0.0, interleaved=False):
    """x [n, heads, D] -> float64; weight, inv_freq may be None."""
    y = x.double().cpu()
    if weight is not None:
        w = weight.double().cpu() + float(torch.tensor(offset, dtype=torch.float32))
        e = float(torch.tensor(eps, dtype=torch.float32))
        y = y * w / torch.sqrt((y * y).mean(-1, keepdim=True) + e)
    if inv_freq is None:
        return y
    half = inv_freq.numel()
    a = positions.double().cpu()[:, None, None] * inv_freq.double().cpu()
    c, s = torch.cos(a), torch.sin(a)
    i = torch.arange(half)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out = y.clone()
    out[..., p] = y[..., p] * c - y[..., q] * s
    out[..., q] = y[..., q] * c + y[..., p] * s
    return out


def rows_bound(ref, dtype):
    """Rounding of the result to its type, and of the fp32 arithmetic: the norm is a few
    roundings (2^-21 covers eight), each of cos and sin is off by at most pi 2^-24 (rounding
    of the reduced angle) plus 2 ulp, against a pair no longer than the row's largest."""
    row = ref.abs().amax(-1, keepdim=True) * math.sqrt(2.0)
    return HALF_STEP[dtype] * ref.abs() * (1 + 2.0 ** -7) + 2.0 ** -20 * row + TINY[dtype]


def gather(cache, k_scale, v_scale, table_row, length):
    """Keys and values [kv_heads, length, D] of one sequence in float64, and which keys lie on
    pages of the cache."""
    ck, cv = cache
    pages, heads, size, D = ck.shape
    key = torch.arange(length)
    ids = table_row.cpu().long()[key // size]
    ok = (ids >= 0) & (ids < pages)
    ids = torch.where(ok, ids, 0)
    used, at = torch.unique(ids, return_inverse=True)
    dev = ck.device
    # 8-bit floats are indexed as bytes
    raw = torch.uint8 if ck.element_size() == 1 else ck.dtype
    kp = ck.view(raw)[used.to(dev)].view(ck.dtype).cpu().double()
    vp = cv.view(raw)[used.to(dev)].view(cv.dtype).cpu().double()
    k = kp[at, :, key % size].transpose(0, 1)
    v = vp[at, :, key % size // 8, :, key % 8].transpose(0, 1)
    if k_scale is not None:
        k = k * k_scale.double().cpu()[:, None, None]
    if v_scale is not None:
        v = v * v_scale.double().cpu()[:, None, None]
    return k, v, ok


def attend(q, cache, k_scale, v_scale, table, lens, starts, scale, window, sinks, two_part):
    """Attention of chunks: q [n, Hq, D], starts [n_seqs + 1]. Returns (out, bound), float64;
    rows outside all sequences are NaN in out. two_part: the probabilities are held as a
    16-bit value plus its 16-bit rest."""
    n, hq, D = q.shape
    dtype = q.dtype
    hkv = cache[0].shape[1]
    G = hq // hkv
    cap = table.shape[1] * cache[0].shape[2]
    out = torch.full((n, hq, D), math.nan, dtype=torch.float64)
    bound = torch.zeros((n, hq, D), dtype=torch.float64)
    q = q.double().cpu()
    scale = float(torch.tensor(scale, dtype=torch.float32))
    half = HALF_STEP[dtype]
    for s in range(len(lens)):
        a, b = starts[s], starts[s + 1]
        L = max(0, min(lens[s], cap))
        m = b - a
        if m == 0:
            continue
        k, v, ok = gather(cache, k_scale, v_scale, table[s], L)
        pos = torch.arange(L - m, L)[:, None]
        key = torch.arange(L)
        seen = (key <= pos) & ok
        if window > 0:
            seen &= (key > pos - window) | (key < sinks)
        for h in range(hq):
            kk, vv = k[h // G], v[h // G]
            x = scale * (q[a:b, h] @ torch.where(seen.any(0)[:, None], kk, 0.0).T)
            x = torch.where(seen, x, -math.inf)
            top = x.amax(-1, keepdim=True) if L else torch.full((m, 1), -math.inf)
            p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
            p = torch.where(seen, p, 0.0)
            total = p.sum(-1, keepdim=True)
            p = p / torch.where(total == 0, 1.0, total)
            finite = torch.where(torch.isfinite(vv), vv, 0.0)
            o = p @ finite
            rough = p @ finite.abs()
            if not torch.isfinite(vv).all():
                # only the rows that see a non-finite value take it
                for j in torch.nonzero(~torch.isfinite(vv).all(-1)).flatten().tolist():
                    add = p[:, j:j + 1] * torch.where(torch.isfinite(vv[j]), 0.0, vv[j])
                    o = o + torch.where(seen[:, j:j + 1], add, 0.0)
            out[a:b, h] = o
            # Rounding of the output; probabilities (one rounding, or two parts: its square);
            # scores: D products and sums in fp32 against sum |q||k|, twice (numerator and
            # denominator); fp32 sums over the keys, exp2 and the scaling (32 roundings);
            # fp16 probabilities below 2^-14 are spaced 2^-24 against a largest of at least 1.
            big = (q[a:b, h].abs() @ torch.where(seen.any(0)[:, None], kk, 0.0).abs().T)
            big = scale * torch.where(seen & torch.isfinite(big), big, 0.0).amax(-1, keepdim=True) \
                if L else torch.zeros((m, 1))
            part = half * half if two_part else half
            slack = part + 2.0 ** -24 * (2 * (D + 8) * big.abs() + L + 32)
            least = L * 2.0 ** -25 * finite.abs().amax(0) if dtype == torch.float16 and L else 0.0
            bound[a:b, h] = half * o.abs() * (1 + 2.0 ** -7) + slack * rough + least + TINY[dtype]
    return out, bound


def assert_close(got, ref, bound, what):
    got = got.double().cpu()
    bad_nan = torch.isnan(got) != torch.isnan(ref)
    assert not bad_nan.any(), f"{what}: NaN at {torch.nonzero(bad_nan)[:4].tolist()}"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities"
    fin = torch.isfinite(ref)
    assert torch.isfinite(got[fin]).all(), f"{what}: not finite"
    d = (got - ref).abs()[fin]
    over = d > bound[fin]
    if over.any():
        i = int(torch.argmax(d / bound[fin]))
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} out of bounds, worst "
                             f"|d| {d[i]:.3e} bound {bound[fin][i]:.3e} ref {ref[fin][i]:.3e}")
