"""Python binding of the microscaled 4-bit products of libqmoe (C ABI in include/qmoe.h):
quantization of rows, products with 4-bit matrices, and the routed-expert layer in them.

Argument marshalling only, as in `qmoe`. The usual calls (no workspace and no stream given,
tensors on the current device) go through a native short path with the same checks;
whatever it does not take is checked and marshalled here. Every call works on the GPU of its tensors (made
current for the call when it is not) and on that GPU's current stream, or on `stream`;
outputs and workspaces that a call makes for itself belong to that stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from .qmoe import (BYTES, F32, FLOATS, MOE_OK, MoeError, Routing, _Args, _current_device,
                   _int, _load_fastcall, _ptr, _raw_stream, _Routing, lib)

_fastcall = _load_fastcall()

BLOCK = 32  # values that share a scale
U8 = (torch.uint8,)


class _MxMatrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32)]


class _MxLayer(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("gate", _MxMatrix), ("up", _MxMatrix), ("down", _MxMatrix)]


def _declare():
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    mat, layer = ctypes.POINTER(_MxMatrix), ctypes.POINTER(_MxLayer)
    lib.moe_mx_quantize.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp]
    lib.moe_mx_dequantize.argtypes = [mat, i64, i32, vp, vp]
    lib.moe_mx_linear_workspace_bytes.argtypes = [i32, i32]
    lib.moe_mx_linear_workspace_bytes.restype = sz
    lib.moe_mx_linear.argtypes = [vp, i32, i64, i32, mat, vp, i32, i64, vp, sz, vp]
    lib.moe_mx_linear_quantized.argtypes = [mat, mat, vp, i32, i64, vp]
    lib.moe_mx_ffn_workspace_bytes.argtypes = [layer, i32]
    lib.moe_mx_ffn_workspace_bytes.restype = sz
    lib.moe_mx_ffn.argtypes = [layer, vp, i32, i64, i32, ctypes.POINTER(_Routing), vp, vp, vp, sz, vp]


_declare()


@dataclass
class MxMatrix:
    """Rows in microscaled 4-bit floats: ``codes`` uint8 ``[..., rows, cols / 2]`` (e2m1, the even
    column in the low half of a byte) and ``scales`` uint8 ``[..., rows, cols / 32]`` (e8m0, the
    exponent + 127; 255: NaN), both contiguous. (Tensors of torch's own 4-bit and scale types
    have these bytes: pass their ``view(torch.uint8)``.)"""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self) -> int:
        return self.codes.shape[-2]

    @property
    def cols(self) -> int:
        return 2 * self.codes.shape[-1]

    @staticmethod
    def empty(*shape: int, device="cuda") -> "MxMatrix":
        """Uninitialised rows of ``shape = (..., rows, cols)``."""
        if len(shape) < 2 or shape[-1] % BLOCK:
            raise ValueError(f"shape: {shape}, expected (..., rows, cols) with cols a multiple of "
                             f"{BLOCK}")
        return MxMatrix(torch.empty((*shape[:-1], shape[-1] // 2), dtype=torch.uint8, device=device),
                        torch.empty((*shape[:-1], shape[-1] // BLOCK), dtype=torch.uint8,
                                    device=device))

    def check(self, name: str, args: _Args, dims: int | None = None, shape=None) -> _MxMatrix:
        args.need(self.codes, f"{name}.codes", U8)
        c = tuple(self.codes.shape)
        if len(c) < 2 or (dims is not None and len(c) != dims):
            raise ValueError(f"{name}.codes: shape {c}, expected {dims or 'at least 2'} axes")
        if self.cols % BLOCK or self.cols == 0:
            raise ValueError(f"{name}: {self.cols} columns, expected a multiple of {BLOCK}")
        if shape is not None and (*c[:-1], self.cols) != tuple(shape):
            raise ValueError(f"{name}: shape {(*c[:-1], self.cols)}, expected {tuple(shape)}")
        args.need(self.scales, f"{name}.scales", U8, shape=(*c[:-1], self.cols // BLOCK))
        return _MxMatrix(self.codes.data_ptr(), self.scales.data_ptr(), _int(self.rows),
                         _int(self.cols))


@dataclass
class MxLayer:
    """A routed-expert layer: gate and up ``[E, d_ff, d_model]``, down ``[E, d_model, d_ff]``."""
    gate: MxMatrix
    up: MxMatrix
    down: MxMatrix
    top_k: int

    def _shape(self) -> tuple[int, int, int]:
        """(experts, d_ff, d_model), as the gate has them."""
        c = self.gate.codes.shape
        if len(c) != 3:
            raise ValueError(f"gate.codes: shape {tuple(c)}, expected [E, d_ff, d_model / 2]")
        return c[0], c[1], 2 * c[2]

    def check(self, args: _Args) -> _MxLayer:
        E, f, d = self._shape()
        return _MxLayer(_int(d), _int(f), _int(E), _int(self.top_k), self.gate.check("gate", args, 3),
                        self.up.check("up", args, 3, (E, f, d)),
                        self.down.check("down", args, 3, (E, d, f)))


class _RowArgs(_Args):
    """Checks of one call's tensors; rows may be a strided view."""

    def rows(self, t, name: str, dtypes, shape=None) -> int:
        """A tensor [n, cols] whose last axis is contiguous; returns its row stride."""
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name}: expected a tensor [n, cols], got "
                             f"{getattr(t, 'shape', type(t))}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(dtypes)}")
        if shape is not None and any(w is not None and w != h for w, h in zip(shape, t.shape)):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: the last axis must be contiguous")
        self.seen.append((name, t))
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]

    def gpu(self) -> torch.device:
        self.on_gpu()
        return self.seen[0][1].device


def _on(device: torch.device, stream):
    """The GPU of the tensors and the stream of the call made current."""
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream: on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _current() -> int:
    return torch.cuda.current_stream().cuda_stream


def _count(n: int, what: str = "rows") -> None:
    if n > 0x7fffffff:  # would not reach the library as it is
        raise ValueError(f"x: {n} {what}")


def _done(fn: str, rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _result(fn: str, r):
    """What a call on the short path returns, or its error."""
    if type(r) is int:
        raise MoeError(fn, r)
    return r


def quantize(x: torch.Tensor, out: MxMatrix | None = None, stream=None) -> MxMatrix:
    """moe_mx_quantize: x ``[..., rows, cols]`` (fp32, bf16 or fp16; contiguous, or two axes with
    a row stride) in 4 bits. A new matrix unless `out` is given."""
    if stream is None and out is None and type(x) is torch.Tensor and x.is_cuda:
        gpu = _current_device()
        r = _fastcall.mx_quantize(gpu, x, _raw_stream(gpu))
        if r is not None:
            return MxMatrix(*_result("moe_mx_quantize", r))
    args = _RowArgs()
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        stride = args.rows(x, "x", FLOATS)
    else:
        args.need(x, "x", tuple(FLOATS))
        if x.dim() < 2:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected [..., rows, cols]")
        stride = x.shape[-1]
    cols = x.shape[-1]
    if cols % BLOCK or cols == 0:
        raise ValueError(f"x: {cols} columns, expected a multiple of {BLOCK}")
    _count(cols, "columns")
    if out is not None:
        out.check("out", args, x.dim(), x.shape)
    device = args.gpu()
    with _on(device, stream):
        if out is None:
            out = MxMatrix.empty(*x.shape, device=device)
        _done("moe_mx_quantize",
              lib.moe_mx_quantize(_ptr(x), FLOATS[x.dtype], x.numel() // cols, cols, stride,
                                  _ptr(out.codes), _ptr(out.scales), _current()))
    return out


def dequantize(m: MxMatrix, dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """moe_mx_dequantize: the values of `m` as fp32, bf16 or fp16 ``[..., rows, cols]``."""
    if stream is None and out is None and m.codes.is_cuda:
        gpu = _current_device()
        r = _fastcall.mx_dequantize(gpu, m.codes, m.scales, FLOATS.get(dtype), _raw_stream(gpu))
        if r is not None:
            return _result("moe_mx_dequantize", r)
    args = _RowArgs()
    st = m.check("m", args)
    if out is not None:
        dtype = out.dtype
        args.need(out, "out", tuple(FLOATS), shape=(*m.codes.shape[:-1], m.cols))
    if dtype not in FLOATS:
        raise ValueError(f"dtype: {dtype}, expected one of {tuple(FLOATS)}")
    device = args.gpu()
    with _on(device, stream):
        if out is None:
            out = torch.empty((*m.codes.shape[:-1], m.cols), dtype=dtype, device=device)
        _done("moe_mx_dequantize",
              lib.moe_mx_dequantize(ctypes.byref(st), m.scales.numel() * BLOCK // m.cols,
                                    FLOATS[dtype], _ptr(out), _current()))
    return out


def linear(x: torch.Tensor | MxMatrix, w: MxMatrix, out: torch.Tensor | None = None,
           dtype: torch.dtype | None = None, ws: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """moe_mx_linear: ``x @ w.T`` with x ``[n, cols]`` quantized on the way, or given as an
    MxMatrix (one quantization then serves several products). w: ``[rows, cols]``. Returns
    ``[n, rows]`` of `dtype` (x's own, bf16 for an MxMatrix, unless `out` or `dtype` is given);
    `out` may have a row stride."""
    quantized = isinstance(x, MxMatrix)
    rows, scales = (x.codes, x.scales) if quantized else (x, None)
    if stream is None and ws is None and type(rows) is torch.Tensor and rows.is_cuda:
        gpu = _current_device()
        to = dtype or (out.dtype if out is not None else torch.bfloat16 if quantized else x.dtype)
        r = _fastcall.mx_linear(gpu, rows, scales, w.codes, w.scales, FLOATS.get(to), out,
                                _raw_stream(gpu))
        if r is not None:
            r = _result("moe_mx_linear_quantized" if quantized else "moe_mx_linear", r)
            return r if out is None else out
    args = _RowArgs()
    wst = w.check("w", args, 2)
    if quantized:
        xst = x.check("x", args, 2)
        if x.cols != w.cols:
            raise ValueError(f"x: {x.cols} columns, expected {w.cols}")
        n = x.rows
    else:
        stride = args.rows(x, "x", FLOATS, (None, w.cols))
        n = x.shape[0]
    _count(n)
    if out is not None:
        if dtype is not None and dtype != out.dtype:
            raise ValueError(f"out: dtype {out.dtype}, expected {dtype}")
        args.rows(out, "out", FLOATS, (n, w.rows))
        dtype = out.dtype
    if dtype is None:
        dtype = torch.bfloat16 if quantized else x.dtype
    if dtype not in FLOATS:
        raise ValueError(f"dtype: {dtype}, expected one of {tuple(FLOATS)}")
    if ws is not None:
        args.need(ws, "ws", BYTES)
    device = args.gpu()
    with _on(device, stream):
        if out is None:
            out = torch.empty((n, w.rows), dtype=dtype, device=device)
        step = out.stride(0) if n > 1 else w.rows
        if quantized:
            _done("moe_mx_linear_quantized",
                  lib.moe_mx_linear_quantized(ctypes.byref(xst), ctypes.byref(wst), _ptr(out),
                                              FLOATS[dtype], step, _current()))
            return out
        if ws is None:
            need = lib.moe_mx_linear_workspace_bytes(n, w.cols)
            ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        _done("moe_mx_linear",
              lib.moe_mx_linear(_ptr(x), FLOATS[x.dtype], stride, n, ctypes.byref(wst), _ptr(out),
                                FLOATS[dtype], step, _ptr(ws), 0 if ws is None else ws.numel(),
                                _current()))
    return out


def ffn_workspace_bytes(layer: MxLayer, n_tokens: int) -> int:
    """Bytes of the workspace of `ffn`; 0 for sizes out of range."""
    E, f, d = layer._shape()
    st = _MxLayer(_int(d), _int(f), _int(E), _int(layer.top_k))
    return int(lib.moe_mx_ffn_workspace_bytes(ctypes.byref(st), _int(n_tokens)))


def ffn(layer: MxLayer, x: torch.Tensor, routing: Routing, residual: torch.Tensor | None = None,
        out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """moe_mx_ffn: the routing-weighted sum of the experts' outputs for x ``[n, d_model]`` (fp32,
    bf16 or fp16), added to `residual` fp32 ``[n, d_model]`` (None: zeros). A new tensor unless
    `out` is given, which may be `residual`."""
    if stream is None and ws is None and type(x) is torch.Tensor and x.is_cuda:
        gpu = _current_device()
        g, u, d = layer.gate, layer.up, layer.down
        r = _fastcall.mx_ffn(gpu, g.codes, g.scales, u.codes, u.scales, d.codes, d.scales, layer.top_k,
                             x, routing.topk_ids, routing.topk_w, routing.expert_offsets,
                             routing.pair_index, residual, out, _raw_stream(gpu))
        if r is not None:
            return out if out is not None and type(r) is not int else _result("moe_mx_ffn", r)
    args = _RowArgs()
    st = layer.check(args)
    stride = args.rows(x, "x", FLOATS, (None, st.d_model))
    n = x.shape[0]
    _count(n)
    routing.check(n, st.n_experts, layer.top_k, args)
    if residual is not None:
        args.need(residual, "residual", F32, shape=(n, st.d_model))
    if out is not None:
        args.need(out, "out", F32, shape=(n, st.d_model))
    if ws is not None:
        args.need(ws, "ws", BYTES)
    device = args.gpu()
    rs = routing._struct()
    with _on(device, stream):
        if out is None:
            out = torch.empty((n, st.d_model), dtype=torch.float32, device=device)
        if ws is None:
            need = lib.moe_mx_ffn_workspace_bytes(ctypes.byref(st), n)
            ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        _done("moe_mx_ffn",
              lib.moe_mx_ffn(ctypes.byref(st), _ptr(x), FLOATS[x.dtype], stride, n, ctypes.byref(rs),
                             _ptr(residual), _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(),
                             _current()))
    return out
