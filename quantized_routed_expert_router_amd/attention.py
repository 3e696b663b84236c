"""Python binding of the attention half of libqmoe (C ABI in include/qmoe.h): norm and
rotation of query and key heads, the paged key-value cache, and attention over it for
decode windows and prefill chunks.

Argument marshalling only, as in `qmoe`. The usual calls (nothing given for outputs,
workspace and stream, tensors on the current device) go through a native short path with
the same checks; whatever it does not take is checked and marshalled here. Every call works on the GPU of its tensors (made
current for the call when it is not) and on that GPU's current stream, or on `stream`;
outputs and workspaces that a call makes for itself belong to that stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from .qmoe import BYTES, F32, I32, MOE_OK, MoeError, _Args, _ptr, lib

try:
    from . import _fastcall
except ImportError as e:
    raise ImportError("_fastcall.so is missing or does not load: build it with "
                      "`python -m quantized_routed_expert_router_amd.build`") from e

MAX_WINDOW_TOKENS = 16
MAX_HEADS = 512

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}
HALF = (torch.bfloat16, torch.float16)
CACHE = (torch.bfloat16, torch.float16, torch.float8_e4m3fn)


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _NormRope(ctypes.Structure):
    _fields_ = [("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _Pages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


class _Attn(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


def _declare():
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    heads, cache = ctypes.POINTER(_Heads), ctypes.POINTER(_KVCache)
    rope, pages, attn = (ctypes.POINTER(c) for c in (_NormRope, _Pages, _Attn))
    lib.moe_qk_norm_rope.argtypes = [heads, heads, vp, i32, i32, i32, rope, heads, heads, vp]
    lib.moe_kv_append.argtypes = [cache, heads, heads, vp, vp, i32, i32, rope, heads, heads, vp]
    lib.moe_attn_decode_workspace_bytes.argtypes = [cache, i32, i32, i32, i32, attn]
    lib.moe_attn_decode_workspace_bytes.restype = sz
    lib.moe_attn_decode.argtypes = [cache, heads, i32, pages, i32, attn, vp, vp, sz, vp]
    lib.moe_attn_prefill_workspace_bytes.argtypes = [cache, i32, i32, i32, i32, attn]
    lib.moe_attn_prefill_workspace_bytes.restype = sz
    lib.moe_attn_prefill.argtypes = [cache, heads, i32, vp, i32, pages, attn, vp, vp, sz, vp]


_declare()


class _HeadArgs(_Args):
    """Checks of one call's tensors; rows of heads may be strided views. Short paths for
    tensors that pass: these calls take a few microseconds on the GPU."""

    def need(self, t, name, dtypes, shape=None, min_numel=None):
        if type(t) is torch.Tensor and min_numel is None and t.dtype in dtypes and \
                t.is_contiguous() and (shape is None or t.shape == shape):
            self.seen.append((name, t))
        else:
            super().need(t, name, dtypes, shape, min_numel)

    def heads(self, t, name: str, dtypes, n=None, heads=None, D=None) -> _Heads:
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name}: expected a tensor [n, heads, head_dim], got "
                             f"{getattr(t, 'shape', type(t))}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
        a, b, c = shape = t.shape
        if (n is not None and a != n) or (heads is not None and b != heads) or \
                (D is not None and c != D):
            raise ValueError(f"{name}: shape {tuple(shape)}, expected "
                             f"{(a if n is None else n, heads or b, D or c)}")
        ts, hs, last = t.stride()
        if last != 1 and c != 1:
            raise ValueError(f"{name}: the last axis must be contiguous")
        self.seen.append((name, t))
        return _Heads(t.data_ptr(), ts, hs, b)

    def table(self, t, name: str, lens) -> _Pages:
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name}: expected a tensor [n_seqs, max_pages], got "
                             f"{getattr(t, 'shape', type(t))}")
        if t.dtype not in I32:
            raise ValueError(f"{name}: dtype {t.dtype}, expected one of {I32}")
        b, most = t.shape
        row, last = t.stride()
        if most > 1 and last != 1:
            raise ValueError(f"{name}: the last axis must be contiguous")
        if b > 1 and row < most:
            raise ValueError(f"{name}: rows overlap")
        self.seen.append((name, t))
        self.need(lens, "kv_lens", I32, (b,))
        return _Pages(t.data_ptr(), lens.data_ptr(), row if b > 1 else most, b, most)

    def gpu(self) -> int:
        """The index of the one GPU that all tensors are on."""
        at = self.seen[0][1].get_device()
        if at < 0:
            self.on_gpu()
        for _, t in self.seen:
            if t.get_device() != at:
                self.on_gpu()
        return at


def _result(fn: str, r):
    """The outputs of a call on the short path, or its error."""
    if type(r) is int:
        raise MoeError(fn, r)
    return r


def _on_stream(fn, args, stream, t):
    """The call with `stream` current, so that what it allocates belongs to that stream."""
    if isinstance(t, torch.Tensor) and t.is_cuda and stream.device != t.device:
        raise ValueError(f"stream: on {stream.device}, the tensors on {t.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = torch.cuda.current_device
_dense = torch.contiguous_format


@dataclass
class KVCache:
    """Paged keys and values of one layer:

    * ``k``: ``[num_pages, kv_heads, page_size, head_dim]``
    * ``v``: ``[num_pages, kv_heads, page_size // 8, head_dim, 8]`` (the last axis is the row
      within a group of 8 rows)

    contiguous, bfloat16, float16 or float8_e4m3fn; the latter hold value / scale with
    `k_scale` and `v_scale` fp32 ``[kv_heads]`` (None: 1)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    @staticmethod
    def empty(num_pages: int, kv_heads: int, page_size: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda", k_scale=None, v_scale=None) -> "KVCache":
        """An uninitialised cache: rows hold anything until they are appended."""
        if page_size % 8:
            raise ValueError(f"page_size: {page_size}, expected a multiple of 8")
        return KVCache(
            torch.empty((num_pages, kv_heads, page_size, head_dim), dtype=dtype, device=device),
            torch.empty((num_pages, kv_heads, page_size // 8, head_dim, 8), dtype=dtype,
                        device=device), k_scale, v_scale)

    def check(self, args: _Args) -> _KVCache:
        k, v = self.k, self.v
        args.need(k, "cache.k", CACHE)
        if k.dim() != 4:
            raise ValueError(f"cache.k: shape {tuple(k.shape)}, expected [num_pages, kv_heads, "
                             "page_size, head_dim]")
        pages, heads, size, D = k.shape
        args.need(v, "cache.v", (k.dtype,), (pages, heads, size // 8, D, 8))
        for name, s in (("cache.k_scale", self.k_scale), ("cache.v_scale", self.v_scale)):
            if s is not None:
                args.need(s, name, F32, (heads,))
        return _KVCache(k.data_ptr(), v.data_ptr(), _ptr(self.k_scale), _ptr(self.v_scale),
                        DTYPES[k.dtype], pages, size, heads, D)


@dataclass
class NormRope:
    """Norm and rotation of head rows (see moe_norm_rope): RMS norm weights fp32
    ``[head_dim]`` of the queries and the keys (None: no norm), rotation frequencies fp32
    ``[rot_dim / 2]`` (None: no rotation)."""
    q_norm: torch.Tensor | None = None
    k_norm: torch.Tensor | None = None
    inv_freq: torch.Tensor | None = None
    eps: float = 1e-6
    weight_offset: float = 0.0
    interleaved: bool = False

    def check(self, D: int, args: _Args) -> _NormRope:
        for name, w in (("q_norm", self.q_norm), ("k_norm", self.k_norm)):
            if w is not None:
                args.need(w, name, F32, (D,))
        rot = 0
        if self.inv_freq is not None:
            args.need(self.inv_freq, "inv_freq", F32)
            rot = 2 * self.inv_freq.numel()
        return _NormRope(_ptr(self.q_norm), _ptr(self.k_norm), _ptr(self.inv_freq), self.eps,
                         self.weight_offset, rot, 1 if self.interleaved else 0)


_ref = ctypes.byref


def _new_heads(like: torch.Tensor):
    t = torch.empty_like(like, memory_format=_dense)
    _, heads, D = like.shape
    return t, _Heads(t.data_ptr(), heads * D, D, heads)


def qk_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None,
                 p: NormRope, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None, stream=None):
    """moe_qk_norm_rope: norm and rotation of query and key heads ``[n, heads, head_dim]``
    (either may be None) at `positions` int32 ``[n]``. Returns (q_out, k_out), new tensors
    unless given; an output may be its own input."""
    if stream is None and q_out is None and k_out is None and type(q) is torch.Tensor and \
            q.is_cuda:
        gpu = _current_device()
        r = _fastcall.qk_norm_rope(gpu, q, k, positions, p.q_norm, p.k_norm, p.inv_freq, p.eps,
                                   p.weight_offset, p.interleaved, _raw_stream(gpu))
        if r is not None:
            return _result("moe_qk_norm_rope", r)
    some = q if q is not None else k
    if some is None:
        raise ValueError("q, k: at least one is needed")
    if stream is not None:
        return _on_stream(qk_norm_rope, (q, k, positions, p, q_out, k_out), stream, some)
    args = _HeadArgs()
    qs = ks = qo = ko = None
    if q is not None:
        qs = args.heads(q, "q", HALF)
    n, D = some.shape[0], some.shape[-1]
    if k is not None:
        ks = args.heads(k, "k", (some.dtype,) if some.dtype in HALF else HALF, n, None, D)
    rope = p.check(D, args)
    if positions is not None:
        args.need(positions, "positions", I32, (n,))
    for name, x, out in (("q_out", q, q_out), ("k_out", k, k_out)):
        if out is not None and x is None:
            raise ValueError(f"{name}: given without its input")
    if q_out is not None:
        qo = args.heads(q_out, "q_out", (some.dtype,), *q.shape)
    if k_out is not None:
        ko = args.heads(k_out, "k_out", (some.dtype,), *k.shape)
    gpu = args.gpu()
    if gpu != _current_device():
        with torch.cuda.device(gpu):
            return qk_norm_rope(q, k, positions, p, q_out, k_out)
    if q is not None and qo is None:
        q_out, qo = _new_heads(q)
    if k is not None and ko is None:
        k_out, ko = _new_heads(k)
    rc = lib.moe_qk_norm_rope(qs and _ref(qs), ks and _ref(ks), _ptr(positions), n,
                              DTYPES[some.dtype], D, _ref(rope), qo and _ref(qo),
                              ko and _ref(ko), _raw_stream(gpu))
    if rc != MOE_OK:
        raise MoeError("moe_qk_norm_rope", rc)
    return q_out, k_out


def kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
              positions: torch.Tensor | None = None, p: NormRope | None = None,
              q: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None):
    """moe_kv_append: k ``[n, kv_heads, head_dim]`` normed and rotated by `p`, and v, into the
    cache at `slots` int32 ``[n]`` (page * page_size + row; outside the cache: not stored).
    With `q`, its heads are normed and rotated in the same launch; returns q_out (a new
    tensor unless given; None without q)."""
    if stream is None and q_out is None and p is not None and type(q) is torch.Tensor and \
            q.is_cuda:
        gpu = _current_device()
        r = _fastcall.kv_append(gpu, cache.k, cache.v, cache.k_scale, cache.v_scale, k, v, slots,
                                positions, p.q_norm, p.k_norm, p.inv_freq, p.eps, p.weight_offset,
                                p.interleaved, q, _raw_stream(gpu))
        if r is not None:
            return _result("moe_kv_append", r)
    if stream is not None:
        return _on_stream(kv_append, (cache, k, v, slots, positions, p, q, q_out), stream, k)
    args = _HeadArgs()
    ks = args.heads(k, "k", HALF)
    n, heads, D = k.shape
    same = (k.dtype,)
    vs = args.heads(v, "v", same, n, heads, D)
    cs = cache.check(args)
    if (cs.kv_heads, cs.head_dim) != (heads, D):
        raise ValueError(f"k: shape {tuple(k.shape)}, the cache has {cs.kv_heads} heads of "
                         f"{cs.head_dim}")
    args.need(slots, "slots", I32, (n,))
    if positions is not None:
        args.need(positions, "positions", I32, (n,))
    rope = p.check(D, args) if p is not None else None
    qs = qo = None
    if q is not None:
        if p is None:
            raise ValueError("q: needs p, its norm and rotation")
        qs = args.heads(q, "q", same, n, None, D)
        if q_out is not None:
            qo = args.heads(q_out, "q_out", same, *q.shape)
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    gpu = args.gpu()
    if gpu != _current_device():
        with torch.cuda.device(gpu):
            return kv_append(cache, k, v, slots, positions, p, q, q_out)
    if q is not None and qo is None:
        q_out, qo = _new_heads(q)
    rc = lib.moe_kv_append(_ref(cs), _ref(ks), _ref(vs), slots.data_ptr(), _ptr(positions), n,
                           DTYPES[k.dtype], rope and _ref(rope), qs and _ref(qs),
                           qo and _ref(qo), _raw_stream(gpu))
    if rc != MOE_OK:
        raise MoeError("moe_kv_append", rc)
    return q_out


def _attn(scale, window: int, sinks: int, D: int) -> _Attn:
    if not 0 <= window < 1 << 31 or not 0 <= sinks < 1 << 31:
        raise ValueError(f"window, sinks: {window}, {sinks}, expected 0..2^31-1")
    return _Attn(D ** -0.5 if scale is None else scale, window, sinks)


def decode_workspace_bytes(cache: KVCache, q_heads: int, n_seqs: int, window_tokens: int,
                           max_pages: int, window: int = 0, sinks: int = 0) -> int:
    """moe_attn_decode_workspace_bytes: workspace of attn_decode calls of these sizes."""
    cs = cache.check(_HeadArgs())
    return lib.moe_attn_decode_workspace_bytes(_ref(cs), q_heads, n_seqs, window_tokens,
                                               max_pages, _ref(_attn(1.0, window, sinks, 1)))


def prefill_workspace_bytes(cache: KVCache, q_heads: int, n_seqs: int, n_tokens: int,
                            max_pages: int, window: int = 0, sinks: int = 0) -> int:
    """moe_attn_prefill_workspace_bytes: workspace of attn_prefill calls of these sizes."""
    cs = cache.check(_HeadArgs())
    return lib.moe_attn_prefill_workspace_bytes(_ref(cs), q_heads, n_seqs, n_tokens, max_pages,
                                                _ref(_attn(1.0, window, sinks, 1)))


def _attend(cache, q, q_starts, page_table, kv_lens, scale, window, sinks, out, ws):
    if out is None and ws is None and type(q) is torch.Tensor and q.is_cuda:
        gpu = _current_device()
        r = _fastcall.attend(gpu, cache.k, cache.v, cache.k_scale, cache.v_scale, q, q_starts,
                             page_table, kv_lens, q.shape[-1] ** -0.5 if scale is None else scale,
                             window, sinks, _raw_stream(gpu))
        if r is not None:
            return _result("moe_attn_decode" if q_starts is None else "moe_attn_prefill", r)
    args = _HeadArgs()
    qs = args.heads(q, "q", HALF)
    n, heads, D = q.shape
    cs = cache.check(args)
    if cs.head_dim != D:
        raise ValueError(f"q: head_dim {D}, the cache has {cs.head_dim}")
    pages = args.table(page_table, "page_table", kv_lens)
    b = pages.n_seqs
    attn = _attn(scale, window, sinks, D)
    prefill = q_starts is not None
    if prefill:
        args.need(q_starts, "q_starts", I32, (b + 1,))
        size = n
    else:
        size = n // b if b else 0
        if size * b != n:
            raise ValueError(f"q: {n} tokens, expected a multiple of {b} sequences")
    if out is not None:
        args.need(out, "out", (q.dtype,), q.shape)
    if ws is not None:
        args.need(ws, "ws", BYTES)
    gpu = args.gpu()
    if gpu != _current_device():
        with torch.cuda.device(gpu):
            return _attend(cache, q, q_starts, page_table, kv_lens, scale, window, sinks, out, ws)
    if out is None:
        out = torch.empty_like(q, memory_format=_dense)
    if n == 0:
        return out
    if ws is None:
        query = (lib.moe_attn_prefill_workspace_bytes if prefill
                 else lib.moe_attn_decode_workspace_bytes)
        room = query(_ref(cs), heads, b, size, pages.max_pages, _ref(attn))
        if room:
            ws = q.new_empty(room, dtype=torch.uint8)
    else:
        room = ws.numel()
    at = ws.data_ptr() if room else None
    if prefill:
        rc = lib.moe_attn_prefill(_ref(cs), _ref(qs), DTYPES[q.dtype], q_starts.data_ptr(), n,
                                  _ref(pages), _ref(attn), out.data_ptr(), at, room,
                                  _raw_stream(gpu))
    else:
        rc = lib.moe_attn_decode(_ref(cs), _ref(qs), DTYPES[q.dtype], _ref(pages), size,
                                 _ref(attn), out.data_ptr(), at, room, _raw_stream(gpu))
    if rc != MOE_OK:
        raise MoeError("moe_attn_prefill" if prefill else "moe_attn_decode", rc)
    return out


def attn_decode(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
                scale: float | None = None, window: int = 0, sinks: int = 0,
                out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """moe_attn_decode: attention of the newest tokens of each sequence. q
    ``[n_seqs * tokens, heads, head_dim]``, sequence-major, the same number of tokens (1..16)
    of each; page_table int32 ``[n_seqs, max_pages]``; kv_lens int32 ``[n_seqs]``, the new
    tokens included. scale: 1/sqrt(head_dim) unless given. Returns out."""
    if stream is not None:
        return _on_stream(attn_decode, (cache, q, page_table, kv_lens, scale, window, sinks, out,
                                        ws), stream, q)
    return _attend(cache, q, None, page_table, kv_lens, scale, window, sinks, out, ws)


def attn_prefill(cache: KVCache, q: torch.Tensor, q_starts: torch.Tensor,
                 page_table: torch.Tensor, kv_lens: torch.Tensor, scale: float | None = None,
                 window: int = 0, sinks: int = 0, out: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, stream=None):
    """moe_attn_prefill: causal attention of prompt chunks. q ``[n, heads, head_dim]``,
    q_starts int32 ``[n_seqs + 1]``: sequence s has tokens q_starts[s] .. q_starts[s+1]-1, the
    last of its kv_lens[s] keys. Rows from q_starts[n_seqs] on are not written. Returns out."""
    if q_starts is None:
        raise ValueError("q_starts: expected a tensor [n_seqs + 1]")
    if stream is not None:
        return _on_stream(attn_prefill, (cache, q, q_starts, page_table, kv_lens, scale, window,
                                         sinks, out, ws), stream, q)
    return _attend(cache, q, q_starts, page_table, kv_lens, scale, window, sinks, out, ws)
