"""The attention-half operators as measured work: cases, inputs, plain forms and 64-bit values.

Four operators of the decoder layer's attention half:

* ``norm_rope``: RMS norm of every query and key head with the position rotation;
* ``append``: keys (normed and rotated) and values written into a paged cache, the queries
  normed and rotated beside them;
* ``decode``: attention of the newest tokens of each sequence over the paged cache;
* ``prefill``: causal attention of prompt chunks over the paged cache, optionally with a
  sliding window and first tokens that stay visible.

Cache layouts: K ``[page][kv head][page_size][D]``, V ``[page][kv head][page_size/8][D][8]``.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
EPS = 1e-6
BASE = 1e6


def listed():
    return [
        # a verify window of 4 tokens of one sequence, far into its context: latency
        dict(name="norm_rope_t4_d256", op="norm_rope", n=4, hq=16, hkv=2, d=256, rot=64, inter=False,
             dtype="bf16", first=200000),
        # the largest prefill chunk, full rotation
        dict(name="norm_rope_8192_d128", op="norm_rope", n=8192, hq=32, hkv=8, d=128, rot=128,
             inter=False, dtype="bf16", first=0),
        # an odd chunk, neighbouring pairs, half precision
        dict(name="norm_rope_1021_d64_f16", op="norm_rope", n=1021, hq=24, hkv=4, d=64, rot=64,
             inter=True, dtype="f16", first=7777),
        # a verify window of one sequence into 16-token pages
        dict(name="append_t4_d128", op="append", n=4, run=4, hq=32, hkv=8, d=128, rot=128, inter=False,
             dtype="bf16", cdtype="bf16", page=16, slots=1024, first=200000),
        # 64 sequences, 4 tokens each, into an 8-bit cache
        dict(name="append_64xt4_e4m3", op="append", n=256, run=4, hq=32, hkv=8, d=128, rot=64,
             inter=False, dtype="bf16", cdtype="e4m3", page=64, slots=8192, first=5000),
        # the largest prefill chunk of one prompt, wide heads
        dict(name="append_8192_d256", op="append", n=8192, run=8192, hq=16, hkv=2, d=256, rot=64,
             inter=False, dtype="bf16", cdtype="bf16", page=32, slots=16384, first=0),
        # one token of a short conversation: latency
        dict(name="decode_1x517", op="decode", b=1, t=1, hq=32, hkv=8, d=128, dtype="bf16",
             cdtype="bf16", page=16, short=517, long=517, window=0, sinks=0),
        # a verify window at the end of a 262144-token context
        dict(name="decode_t4_262144_d256", op="decode", b=1, t=4, hq=16, hkv=2, d=256, dtype="bf16",
             cdtype="bf16", page=64, short=262144, long=262144, window=0, sinks=0),
        # 64 conversations of very different lengths, 8-bit cache in small pages
        dict(name="decode_64_ragged_e4m3", op="decode", b=64, t=1, hq=32, hkv=8, d=128, dtype="bf16",
             cdtype="e4m3", page=16, short=1, long=32768, window=0, sinks=0),
        # a short prompt on its own
        dict(name="prefill_37_d64_f16", op="prefill", b=1, q=37, ctx=0, hq=16, hkv=4, d=64, dtype="f16",
             cdtype="f16", page=16, window=0, sinks=0),
        # the largest prefill chunk, at the start of a prompt
        dict(name="prefill_8192_d128", op="prefill", b=1, q=8192, ctx=0, hq=32, hkv=8, d=128,
             dtype="bf16", cdtype="bf16", page=64, window=0, sinks=0),
        # two uneven chunks deep in their prompts, sliding window and first tokens
        dict(name="prefill_window_2x1999", op="prefill", b=2, q=1999, ctx=30000, hq=32, hkv=8, d=128,
             dtype="bf16", cdtype="bf16", page=32, window=4096, sinks=4, ),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "prefill"])
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["bf16", "f16"])
    cdtype = rng.choice([dtype, dtype, "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    hq = hkv * group
    if op in ("norm_rope", "append"):
        # never more elements than the largest chunk
        n = _log(rng, 1, min(8192, 8192 * 5120 // ((hq + 2 * hkv) * d)))
        rot = rng.choice([d, d, d // 2, d // 4])
        case = dict(op=op, n=n, hq=hq, hkv=hkv, d=d, rot=rot, inter=rng.random() < 0.3, dtype=dtype,
                    first=rng.randrange(0, 250000))
        if op == "append":
            case.update(run=rng.choice([1, 2, 4, 5, n]), cdtype=cdtype, page=page,
                        slots=-(-(2 * n + 64) // page) * page)
            case["run"] = min(case["run"], n)
        return case
    window = rng.choice([0, 0, _log(rng, 16, 8192)])
    sinks = rng.choice([0, 4, 17]) if window else 0
    if op == "decode":
        b = _log(rng, 1, 64)
        t = min(rng.choice([1, 1, 2, 4, 5, 8]), 512 // b)
        # no more cache elements than 64 sequences of 16384 tokens, 8 heads of 128
        most = min(262144, (1 << 30) // (b * hkv * d * (1 if cdtype == "e4m3" else 2)))
        long = _log(rng, t, most)
        short = rng.choice([long, max(1, long // 7), 1])
        return dict(op=op, b=b, t=t, hq=hq, hkv=hkv, d=d, dtype=dtype, cdtype=cdtype, page=page,
                    short=short, long=long, window=window, sinks=sinks)
    b = rng.choice([1, 1, 2, 3, 7])
    q = _log(rng, 1, 8192 // b)
    most = max(1, min(65536, (1 << 30) // (b * hq * q)) - q)
    ctx = rng.choice([0, _log(rng, 1, most)])
    return dict(op=op, b=b, q=q, ctx=ctx, hq=hq, hkv=hkv, d=d, dtype=dtype, cdtype=cdtype, page=page,
                window=window, sinks=sinks)


def _lens(case):
    """Query and key counts of each sequence (a function of the case alone)."""
    b = case["b"]
    if case["op"] == "decode":
        lo, hi = case["short"], case["long"]
        return [case["t"]] * b, [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]
    # the first chunk is the longest; the others get shorter, down to about a third
    q = [max(1, case["q"] - case["q"] * 2 * i // (3 * max(1, b - 1))) if i else case["q"] for i in range(b)]
    ctx = [case["ctx"] - case["ctx"] * i // (2 * b) for i in range(b)]
    return q, [x + c for x, c in zip(q, ctx)]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def normal(shape, dtype=dt, scale=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if dtype == torch.float32
                           else torch.bfloat16).mul_(scale).to(dtype)

    s = dict(case=case)
    if case["op"] in ("norm_rope", "append"):
        n, rot = case["n"], case["rot"]
        # one fused projection output, split into heads without a copy
        qkv = normal((n, (hq + 2 * hkv) * d))
        s["q"] = qkv[:, : hq * d].view(n, hq, d)
        s["k"] = qkv[:, hq * d: (hq + hkv) * d].view(n, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(n, hkv, d)
        s["q_norm"] = 1 + normal((d,), torch.float32, 0.1)
        s["k_norm"] = 1 + normal((d,), torch.float32, 0.1)
        s["inv_freq"] = (BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)).float()
        # runs of consecutive positions, one run a sequence
        at = torch.arange(n, device=dev)
        run_len = case.get("run", n)
        s["positions"] = (case["first"] + at % run_len + 31 * (at // run_len)).to(torch.int32)
    if case["op"] == "append":
        page, slots = case["page"], case["slots"]
        pages = slots // page
        ct = TYPES[case["cdtype"]]
        s["ck"] = normal((pages, hkv, page, d), ct)
        s["cv"] = normal((pages, hkv, page // 8, d, 8), ct)
        if case["cdtype"] == "e4m3":
            s["k_scale"] = 0.02 + 0.01 * torch.rand(hkv, generator=g, device=dev)
            s["v_scale"] = 0.02 + 0.01 * torch.rand(hkv, generator=g, device=dev)
        # each run goes to consecutive slots of its own stretch, pages in a shuffled order
        per = slots // (-(-n // run_len))
        logical = (at // run_len) * per + (at % run_len)
        order = torch.randperm(pages, generator=g, device=dev)
        s["slots"] = (order[logical // page] * page + logical % page).to(torch.int32)
    if case["op"] in ("decode", "prefill"):
        qlens, lens = _lens(case)
        page = case["page"]
        most = max(1, -(-max(lens) // page))
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 3
        ct = TYPES[case["cdtype"]]
        s["q"] = normal((sum(qlens), hq, d))
        s["ck"] = normal((pages, hkv, page, d), ct)
        s["cv"] = normal((pages, hkv, page // 8, d, 8), ct)
        if case["cdtype"] == "e4m3":
            s["k_scale"] = 0.5 + torch.rand(hkv, generator=g, device=dev)
            s["v_scale"] = 0.5 + torch.rand(hkv, generator=g, device=dev)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros((len(lens), most), dtype=torch.int32, device=dev)
        at = 0
        for i, m in enumerate(need):
            table[i, :m] = order[at: at + m]
            at += m
        s["table"] = table
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        ends = [sum(qlens[:i]) for i in range(len(qlens) + 1)]
        s["starts"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["most_q"] = max(qlens)
    return s


def _turn(x, weight, positions, inv_freq, interleaved):
    """Norm of each head and rotation, in 32 bits (the angles in 64)."""
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    angle = positions.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = inv_freq.numel()
    if interleaved:
        a, b = y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half: 2 * half]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1)


def _held(x, like, scale):
    """Values as the cache holds them."""
    if like == torch.float8_e4m3fn:
        x = (x.float() / scale[:, None]).clamp(-448.0, 448.0)
    return x.to(like)


def _attend(s, most_q, window, sinks):
    """Attention of every sequence at once, padded to the longest, in 32 bits."""
    q, ck, cv, table, lens, starts = (s[x] for x in ("q", "ck", "cv", "table", "lens", "starts"))
    n, hq, d = q.shape
    b, hkv = table.shape[0], ck.shape[1]
    dev = q.device
    counts = starts[1:] - starts[:-1]
    at = torch.arange(most_q, device=dev)
    rows = (starts[:-1, None] + at).clamp(max=n - 1).long()
    qp = q[rows].float().view(b, most_q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    qp = qp.reshape(b * hkv, -1, d)
    pages = table.long()
    k = ck[pages].float().permute(0, 2, 1, 3, 4).reshape(b * hkv, -1, d)
    v = cv[pages].float().permute(0, 2, 1, 3, 5, 4).reshape(b * hkv, -1, d)
    if "k_scale" in s:
        k = k * s["k_scale"].repeat(b)[:, None, None]
        v = v * s["v_scale"].repeat(b)[:, None, None]
    score = (qp @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(d))
    key = torch.arange(k.shape[1], device=dev)
    pos = (lens[:, None] - counts[:, None] + at)[:, :, None]
    seen = (key <= pos) & (key < lens[:, None, None])
    if window > 0:
        seen &= (key > pos - window) | (key < sinks)
    score = score.view(b, hkv, hq // hkv, most_q, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    score /= torch.where(total == 0, 1.0, total)
    out = score.view(b * hkv, -1, k.shape[1]) @ v
    out = out.view(b, hkv, hq // hkv, most_q, d).permute(0, 3, 1, 2, 4).reshape(b, most_q, hq, d)
    row = torch.arange(n, device=dev, dtype=torch.int32)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return out[seq, (row - starts[seq]).long()].to(q.dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from quantized_routed_expert_router_amd import attention as att
        if op == "norm_rope":
            p = att.NormRope(s["q_norm"], s["k_norm"], s["inv_freq"], eps=EPS, interleaved=case["inter"])
            return att.qk_norm_rope(s["q"], s["k"], s["positions"], p)
        cache = att.KVCache(s["ck"], s["cv"], s.get("k_scale"), s.get("v_scale"))
        if op == "append":
            p = att.NormRope(s["q_norm"], s["k_norm"], s["inv_freq"], eps=EPS, interleaved=case["inter"])
            q = att.kv_append(cache, s["k"], s["v"], s["slots"], s["positions"], p, q=s["q"])
            return q, s["ck"], s["cv"]
        if op == "decode":
            return att.attn_decode(cache, s["q"], s["table"], s["lens"], window=case["window"],
                                   sinks=case["sinks"])
        return att.attn_prefill(cache, s["q"], s["starts"], s["table"], s["lens"],
                                window=case["window"], sinks=case["sinks"])
    if op == "norm_rope":
        q = _turn(s["q"], s["q_norm"], s["positions"], s["inv_freq"], case["inter"])
        k = _turn(s["k"], s["k_norm"], s["positions"], s["inv_freq"], case["inter"])
        return q.to(s["q"].dtype), k.to(s["k"].dtype)
    if op == "append":
        ck, cv = s["ck"], s["cv"]
        q = _turn(s["q"], s["q_norm"], s["positions"], s["inv_freq"], case["inter"]).to(s["q"].dtype)
        k = _turn(s["k"], s["k_norm"], s["positions"], s["inv_freq"], case["inter"])
        slots, page = s["slots"].long(), ck.shape[2]
        to, row = slots // page, slots % page
        # 8-bit floats are indexed through their bytes
        raw = torch.uint8 if ck.dtype == torch.float8_e4m3fn else ck.dtype
        ck.view(raw)[to, :, row] = _held(k, ck.dtype, s.get("k_scale")).view(raw)
        cv.view(raw)[to, :, row // 8, :, row % 8] = _held(s["v"], cv.dtype, s.get("v_scale")).view(raw)
        return q, ck, cv
    return _attend(s, s["most_q"], case["window"], case["sinks"])


def _pairs(case):
    """Visible (query, key) pairs, and the keys that any query of a sequence sees."""
    pairs = keys = 0
    window, sinks = case["window"], case["sinks"]
    for m, length in zip(*_lens(case)):
        lo = None
        for p in range(max(0, length - m), length):
            if window > 0:
                first = max(0, p - window + 1)
                pairs += p + 1 - first + min(sinks, first)
                lo = first if lo is None else lo
            else:
                pairs += p + 1
                lo = 0
        if lo is not None:
            keys += length - lo + min(sinks, lo)
    return pairs, keys


def work(case):
    hq, hkv, d, e = case["hq"], case["hkv"], case["d"], SIZE[case["dtype"]]
    if case["op"] == "norm_rope":
        elements = case["n"] * (hq + hkv) * d
        return {"bytes": 2 * elements * e + 4 * case["n"], "flops": 10 * elements}
    if case["op"] == "append":
        n = case["n"]
        moved = n * d * (2 * hq * e + 2 * hkv * (e + SIZE[case["cdtype"]]))
        return {"bytes": moved + 8 * n, "flops": 10 * n * (hq + hkv) * d}
    pairs, keys = _pairs(case)
    rows = sum(_lens(case)[0])
    return {"bytes": 2 * keys * hkv * d * SIZE[case["cdtype"]] + 2 * rows * hq * d * e + 4 * -(-keys // case["page"]),
            "flops": 4 * pairs * hq * d}


def _rotated64(x, weight, positions, inv_freq, interleaved):
    """Each pair of coordinates as a complex number times e^(i angle), in 64 bits."""
    x = x.double()
    x = weight.double() * x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    m = inv_freq.numel()
    out = x.clone()
    first, second = (slice(0, 2 * m, 2), slice(1, 2 * m, 2)) if interleaved else (slice(0, m), slice(m, 2 * m))
    angle = torch.outer(positions.double(), inv_freq.double()).unsqueeze(1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
    out[..., first], out[..., second] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_rope", "append"):
        q = _rotated64(s["q"], s["q_norm"], s["positions"], s["inv_freq"], case["inter"])
        k = _rotated64(s["k"], s["k_norm"], s["positions"], s["inv_freq"], case["inter"])
        if case["op"] == "norm_rope":
            return q, k
        v = s["v"].double()
        if case["cdtype"] == "e4m3":
            k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
            v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
        ck, cv = s["ck"].double(), s["cv"].double()
        page = ck.shape[2]
        flat = ck.transpose(1, 2).reshape(-1, *k.shape[1:])  # [slot][head][d]
        flat[s["slots"].long()] = k
        ck = flat.view(ck.shape[0], page, *k.shape[1:]).transpose(1, 2)
        flat = cv.permute(0, 2, 4, 1, 3).reshape(-1, *v.shape[1:])
        flat[s["slots"].long()] = v
        cv = flat.view(cv.shape[0], page // 8, 8, *v.shape[1:]).permute(0, 3, 1, 4, 2)
        return q, ck, cv
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    qlens, lens = _lens(case)
    base = 0
    for i, (m, length) in enumerate(zip(qlens, lens)):
        slot = torch.arange(length, device=out.device)
        pg = s["table"][i].long()[slot // page]
        for h in range(hkv):
            k = s["ck"][:, h][pg, slot % page].double()
            v = s["cv"][:, h][pg, slot % page // 8, :, slot % 8].double()
            if case["cdtype"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for r0 in range(0, m, 512):
                r1 = min(m, r0 + 512)
                pos = torch.arange(length - m + r0, length - m + r1, device=out.device)
                hidden = slot > pos[:, None]
                if case["window"] > 0:
                    hidden |= (slot <= pos[:, None] - case["window"]) & (slot >= case["sinks"])
                qs = s["q"][base + r0: base + r1, h * group: (h + 1) * group].double()
                a = torch.einsum("rgd,jd->rgj", qs, k) / math.sqrt(d)
                a = a.masked_fill(hidden[:, None], -math.inf)
                p = torch.softmax(a, -1).masked_fill(hidden[:, None], 0.0)
                out[base + r0: base + r1, h * group: (h + 1) * group] = torch.einsum("rgj,jd->rgd", p, v)
        base += m
    return out
