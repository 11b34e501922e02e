"""Between a language model's body and its loss, in 8 bits: RMS norm of a
residual stream, activations kept in 8 bits for the backward pass, and products
of 8-bit integers.

Thin marshalling over the C ABI (include/sgc.h), as in ``lm``, whose
conventions hold here too: 2-D tensors with contiguous rows at any stride,
gradients as explicit calls, a tensor that requires grad refused while grad
mode is on.  Rows in 8 bits travel as ``Quantized``: what ``rms_norm_q8`` and
``quantize_q8`` give, the backward calls and ``int8_linear`` take.  Calls run
on the tensors' device, whichever is current.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from functools import lru_cache
from typing import Optional

import torch

from . import _check, lib
from .lm import (_DTYPES, NORM_ADD_GRADS, NormOpts, _affine, _empty, _no_graph, _ptr, _rows, _scratch, _vec1,
                 _written)

NORM_LAYER, NORM_RMS = 0, 1
Q8_GROUPS = (0, 32, 64, 128, 256)


class Q8Opts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("dtype", C.c_int32), ("group", C.c_int32)]


class NormQ8Opts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("dtype", C.c_int32), ("wdtype", C.c_int32),
                ("group", C.c_int32), ("kind", C.c_int32), ("flags", C.c_int32), ("reserved", C.c_int32)]


class Int8Opts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("width", C.c_int64), ("out", C.c_int64), ("dtype", C.c_int32),
                ("reserved", C.c_int32)]


def _declare(L) -> None:
    P, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
    for name, args, res in (
            ("sgc_rms_norm", [P, P, i64, P, i64, P, P, i64, P, i64, P, i64, P, P, P], C.c_int),
            ("sgc_rms_norm_backward_workspace", [P], sz),
            ("sgc_rms_norm_backward", [P, P, i64, P, i64, P, P, P, i64, P, i64, P, P, sz, P], C.c_int),
            ("sgc_quantize_q8", [P, P, i64, P, i64, P, P], C.c_int),
            ("sgc_dequantize_q8", [P, P, i64, P, P, i64, P], C.c_int),
            ("sgc_norm_backward_q8_workspace", [P], sz),
            ("sgc_norm_backward_q8", [P, P, i64, P, i64, P, P, P, P, P, P, i64, P, i64, P, i64, P, P, P, sz, P],
             C.c_int),
            ("sgc_int8_linear", [P, P, i64, P, P, i64, P, P, P, i64, P], C.c_int)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


def _run(name: str, device: torch.device, stream, *args) -> None:
    """Calls the library with the device of the tensors current."""
    f = getattr(lib(), name)
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = f(*args, handle)
    if rc:
        _check(rc, name)


def _like(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """Checks rows of a known shape, type and device; their stride."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must match the input's shape, type and device")
    stride = t.stride()
    if stride[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return stride[0]


# ------------------------------------------------------------- 8 bits
@dataclass
class Quantized:
    """Rows in 8 bits: q * scale, a scale every `group` elements of a row (0: one a row)."""
    q: torch.Tensor      # int8 [rows, cols], any row stride
    scale: torch.Tensor  # float32 [rows, groups of a row]
    group: int = 0


def _groups(cols: int, group: int) -> int:
    if group not in Q8_GROUPS:
        raise ValueError(f"group must be one of {Q8_GROUPS}")
    return -(-cols // group) if group else 1


def _q8(t: Quantized, name: str):
    """Checks 8-bit rows; their number, length and stride."""
    q, scale, group = t.q, t.scale, t.group
    if not q.is_cuda:
        raise ValueError(f"{name}.q must be a device (HIP) tensor")
    if q.dim() != 2 or q.dtype != torch.int8:
        raise ValueError(f"{name}.q must be 2-D int8")
    rows, cols = q.shape
    stride = q.stride()
    if stride[1] != 1 and cols > 1:
        raise ValueError(f"{name}.q must have contiguous rows")
    shape = (rows, _groups(cols, group) if group else 1)
    if scale.shape != shape or scale.dtype != torch.float32 or scale.device != q.device or not scale.is_contiguous():
        raise ValueError(f"{name}.scale must be a contiguous float32 tensor of shape {shape} on {q.device}")
    return rows, cols, stride[0]


def _q8_like(t: Quantized, name: str, rows: int, cols: int, device) -> int:
    """_q8 for rows of a known number, length and device; their stride."""
    n, c, stride = _q8(t, name)
    if n != rows or c != cols or t.q.device != device:
        raise ValueError(f"{name}.q must match the call's shape and device")
    return stride


def _new_q8(stream, rows: int, cols: int, group: int, device) -> Quantized:
    """Rows that begin at multiples of 16 bytes, which the products read fastest."""
    whole = -(-cols // 16) * 16
    q = _empty(stream, (rows, whole), torch.int8, device)
    return Quantized(q if whole == cols else q[:, :cols],
                     _empty(stream, (rows, _groups(cols, group) if group else 1), torch.float32, device), group)


def quantize_q8(x: torch.Tensor, *, group: int = 128, out: Optional[Quantized] = None, stream=None) -> Quantized:
    """Rows of x in 8 bits, a scale every `group` elements (32, 64, 128, 256), or one a row (0): activations kept
    for the backward pass; weights, which int8_linear reads (group 0)."""
    _no_graph(x, None if out is None else out.scale)
    xs = _rows(x, "x")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        to = _new_q8(stream, rows, cols, group, dev)
        qs = to.q.stride(0)
    else:
        to = out
        if out.group != group:
            raise ValueError("out.group must be the call's group")
        qs = _q8_like(out, "out", rows, cols, dev)
    o = Q8Opts(rows, cols, _DTYPES[x.dtype], group)
    _run("sgc_quantize_q8", dev, stream, C.byref(o), _ptr(x), xs, _ptr(to.q), qs, _ptr(to.scale))
    if out is not None:
        _written(out.q, out.scale)
    return to


def dequantize_q8(x: Quantized, dtype: torch.dtype = torch.float32, *, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """The values that 8-bit rows stand for."""
    _no_graph(x.scale, out)
    rows, cols, qs = _q8(x, "x")
    dev = x.q.device
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if out is None:
        to, xs = _empty(stream, (rows, cols), dtype, dev), cols
    else:
        to, xs = out, _rows(out, "out")
        if out.shape != x.q.shape or out.dtype != dtype or out.device != dev:
            raise ValueError("out must match the rows' shape and device and the type asked for")
    o = Q8Opts(rows, cols, _DTYPES[dtype], x.group)
    _run("sgc_dequantize_q8", dev, stream, C.byref(o), _ptr(x.q), qs, _ptr(x.scale), _ptr(to), xs)
    _written(out)
    return to


# ----------------------------------------------------------------- RMS norm
@dataclass
class RmsNormalized:
    y: torch.Tensor
    sum: torch.Tensor    # the residual stream after the addition; x where there is none (a copy where y is in x)
    rstd: torch.Tensor   # float32 [rows]


@dataclass
class RmsQuantized:
    q8: Quantized        # the normed rows, one scale a row
    sum: torch.Tensor
    rstd: torch.Tensor


@dataclass
class RmsGrads:
    dx: Optional[torch.Tensor]        # of the stream: of x and of the residual
    dweight: Optional[torch.Tensor]   # float32 [cols]


def _rms(x, weight, residual, sum_out, out, eps, eight, stream):
    """Either kind of output: y (out a tensor), or with `eight` Quantized; the sum, rstd."""
    if torch.is_grad_enabled():
        _no_graph(x, weight, residual, sum_out, out.scale if eight and out is not None else out)
    xs = _rows(x, "x")
    rows, cols = x.shape
    dev, dt = x.device, x.dtype
    wdt = _affine(weight, None, x, cols, dev)
    rs = ss = ys = qs = 0
    y = q8 = total = None
    if residual is not None:
        rs = _like(residual, "residual", x.shape, dt, dev)
    if eight:
        if out is None:
            q8 = _new_q8(stream, rows, cols, 0, dev)
            qs = q8.q.stride(0)
        else:
            if out.group:
                raise ValueError("out must have one scale a row (group 0)")
            q8, qs = out, _q8_like(out, "out", rows, cols, dev)
    elif out is None:
        y, ys = _empty(stream, (rows, cols), dt, dev), cols
    else:
        y, ys = out, _like(out, "out", x.shape, dt, dev)
    if sum_out is not None:
        total, ss = sum_out, _like(sum_out, "sum_out", x.shape, dt, dev)
    elif residual is not None or (y is not None and y.data_ptr() == x.data_ptr()):
        # without a residual the stream is x, unless y takes its place
        total, ss = _empty(stream, (rows, cols), dt, dev), cols
    rstd = _empty(stream, (rows,), torch.float32, dev)
    o = NormOpts(rows, cols, _DTYPES[dt], wdt, eps, 0)
    _run("sgc_rms_norm", dev, stream, C.byref(o), x.data_ptr(), xs, _ptr(residual), rs, _ptr(weight), _ptr(total), ss,
         _ptr(y), ys, q8.q.data_ptr() if eight else None, qs, q8.scale.data_ptr() if eight else None,
         rstd.data_ptr())
    if sum_out is not None:
        _written(sum_out)
    if out is not None:
        _written(*((out.q, out.scale) if eight else (out,)))
    return q8 if eight else y, x if total is None else total, rstd


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
             stream=None) -> RmsNormalized:
    """RMS norm of every row of x + residual [rows, cols]; the sum, rounded to
    x's type, is given too.  out and sum_out may be x or residual, not the
    same one.  Where out is x and there is no residual, x as it was is copied
    into sum."""
    return RmsNormalized(*_rms(x, weight, residual, sum_out, out, eps, False, stream))


def rms_norm_q8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, residual: Optional[torch.Tensor] = None,
                eps: float = 1e-6, out: Optional[Quantized] = None, sum_out: Optional[torch.Tensor] = None,
                stream=None) -> RmsQuantized:
    """rms_norm with its output in 8 bits, a scale a row: what int8_linear takes."""
    return RmsQuantized(*_rms(x, weight, residual, sum_out, out, eps, True, stream))


@lru_cache(maxsize=1024)
def rms_norm_backward_workspace_bytes(rows: int, cols: int, dtype: torch.dtype = torch.float32) -> int:
    """Workspace bytes of one rms_norm_backward call; 0 for sizes that it refuses."""
    return int(lib().sgc_rms_norm_backward_workspace(
        C.byref(NormOpts(rows, cols, _DTYPES[dtype], _DTYPES[torch.float32], 0.0, 0))))


def rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor, *,
                      dsum: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                      dweight: Optional[torch.Tensor] = None, accumulate: bool = False, want_dx: bool = True,
                      ws: Optional[torch.Tensor] = None, stream=None) -> RmsGrads:
    """Gradients of rms_norm at the stream s (the forward call's sum).  dsum is
    the gradient that reaches the stream past the norm.  dweight (float32, e.g.
    a slice of a flat gradient) is written, or with accumulate added to.  dx
    may be dy, s or dsum."""
    if torch.is_grad_enabled():
        _no_graph(dy, s, weight, rstd, dsum, dx, dweight)
    ss = _rows(s, "s")
    shape, dt, dev = s.shape, s.dtype, s.device
    rows, cols = shape
    dys = _like(dy, "dy", shape, dt, dev)
    wdt = _affine(weight, None, s, cols, dev)
    _vec1(rstd, "rstd", rows, torch.float32, dev)
    dss = 0 if dsum is None else _like(dsum, "dsum", shape, dt, dev)
    if accumulate and dweight is None:
        raise ValueError("accumulate needs dweight")
    given, dxs = (dx, dweight), cols
    if dx is not None:
        dxs = _like(dx, "dx", shape, dt, dev)
    elif want_dx:
        dx = _empty(stream, (rows, cols), dt, dev)
    if dweight is None:
        dweight = _empty(stream, (cols,), torch.float32, dev)
    else:
        _vec1(dweight, "dweight", cols, torch.float32, dev)
    o = NormOpts(rows, cols, _DTYPES[dt], wdt, 0.0, NORM_ADD_GRADS if accumulate else 0)
    need = rms_norm_backward_workspace_bytes(rows, cols, dt)
    if ws is not None:
        need = ws.numel() * ws.element_size()
    ws = _scratch(need, ws, dev, "rms_norm", stream, "sgc_rms_norm_backward_workspace")
    _run("sgc_rms_norm_backward", dev, stream, C.byref(o), dy.data_ptr(), dys, s.data_ptr(), ss, _ptr(weight),
         rstd.data_ptr(), _ptr(dsum), dss, _ptr(dx), dxs, dweight.data_ptr(), ws.data_ptr(), need)
    _written(*given)
    return RmsGrads(dx, dweight)


# ------------------------------------------- norms from activations in 8 bits
@dataclass
class NormQ8Grads:
    dx: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]   # float32 [cols]
    dbias: Optional[torch.Tensor]     # float32 [cols]; None for an RMS norm
    y: Optional[torch.Tensor]         # the norm's output from the 8 bits, where wanted


@lru_cache(maxsize=1024)
def norm_backward_q8_workspace_bytes(rows: int, cols: int, *, kind: int = NORM_RMS, group: int = 128,
                                     dtype: torch.dtype = torch.float32) -> int:
    """Workspace bytes of one rms_norm_backward_q8 (NORM_RMS) or layer_norm_backward_q8 (NORM_LAYER) call."""
    return int(lib().sgc_norm_backward_q8_workspace(
        C.byref(NormQ8Opts(rows, cols, _DTYPES[dtype], _DTYPES[torch.float32], group, kind, 0, 0))))


def _backward_q8(kind, dy, x, weight, bias, mean, rstd, dsum, dx, dweight, dbias, accumulate, want_dx, want_y, y, ws,
                 stream) -> NormQ8Grads:
    if torch.is_grad_enabled():
        _no_graph(dy, x.scale, weight, bias, mean, rstd, dsum, dx, dweight, dbias, y)
    layer = kind == NORM_LAYER
    dys = _rows(dy, "dy")
    shape, dt, dev = dy.shape, dy.dtype, dy.device
    rows, cols = shape
    qs = _q8_like(x, "x", rows, cols, dev)
    wdt = _affine(weight, bias, dy, cols, dev)
    _vec1(mean, "mean", rows, torch.float32, dev)
    _vec1(rstd, "rstd", rows, torch.float32, dev)
    dss = 0 if dsum is None else _like(dsum, "dsum", shape, dt, dev)
    if accumulate and (dweight is None or (layer and dbias is None)):
        raise ValueError("accumulate needs dweight" + (" and dbias" if layer else ""))
    given, dxs, ys = (dx, dweight, dbias, y), cols, cols
    if dx is not None:
        dxs = _like(dx, "dx", shape, dt, dev)
    elif want_dx:
        dx = _empty(stream, (rows, cols), dt, dev)
    if y is not None:
        ys = _like(y, "y", shape, dt, dev)
    elif want_y:
        y = _empty(stream, (rows, cols), dt, dev)
    if dweight is None:
        dweight = _empty(stream, (cols,), torch.float32, dev)
    else:
        _vec1(dweight, "dweight", cols, torch.float32, dev)
    if dbias is not None:
        _vec1(dbias, "dbias", cols, torch.float32, dev)
    elif layer:
        dbias = _empty(stream, (cols,), torch.float32, dev)
    o = NormQ8Opts(rows, cols, _DTYPES[dt], wdt, x.group, kind, NORM_ADD_GRADS if accumulate else 0, 0)
    need = norm_backward_q8_workspace_bytes(rows, cols, kind=kind, group=x.group, dtype=dt)
    if ws is not None:
        need = ws.numel() * ws.element_size()
    ws = _scratch(need, ws, dev, "norm_q8", stream, "sgc_norm_backward_q8_workspace")
    _run("sgc_norm_backward_q8", dev, stream, C.byref(o), dy.data_ptr(), dys, x.q.data_ptr(), qs, x.scale.data_ptr(),
         _ptr(weight), _ptr(bias), _ptr(mean), _ptr(rstd), _ptr(dsum), dss, _ptr(dx), dxs, _ptr(y), ys,
         dweight.data_ptr(), _ptr(dbias), ws.data_ptr(), need)
    _written(*given)
    return NormQ8Grads(dx, dweight, dbias, y)


def rms_norm_backward_q8(dy: torch.Tensor, x: Quantized, weight: Optional[torch.Tensor], rstd: torch.Tensor, *,
                         dsum: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                         dweight: Optional[torch.Tensor] = None, accumulate: bool = False, want_dx: bool = True,
                         want_y: bool = False, y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                         stream=None) -> NormQ8Grads:
    """rms_norm_backward with the stream kept in 8 bits; with want_y (or a
    buffer y) the norm's output too, which the next product's weight gradient
    reads.  dx may be dy or dsum."""
    return _backward_q8(NORM_RMS, dy, x, weight, None, None, rstd, dsum, dx, dweight, None, accumulate, want_dx,
                        want_y, y, ws, stream)


def layer_norm_backward_q8(dy: torch.Tensor, x: Quantized, weight: Optional[torch.Tensor],
                           bias: Optional[torch.Tensor], mean: torch.Tensor, rstd: torch.Tensor, *,
                           dsum: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                           dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                           accumulate: bool = False, want_dx: bool = True, want_y: bool = False,
                           y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                           stream=None) -> NormQ8Grads:
    """layer_norm_backward with the norm's input kept in 8 bits; the rest as in
    rms_norm_backward_q8.  bias is read for y alone."""
    if mean is None:
        raise ValueError("a layer norm's backward pass needs mean")
    return _backward_q8(NORM_LAYER, dy, x, weight, bias, mean, rstd, dsum, dx, dweight, dbias, accumulate, want_dx,
                        want_y, y, ws, stream)


# ------------------------------------------------------ products in 8 bits
def int8_linear(x: Quantized, w: Quantized, bias: Optional[torch.Tensor] = None, *,
                dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Product of rows in 8 bits [rows, width] with weights in 8 bits [out,
    width], each with one scale a row, plus bias [out] float32.  For scoring and
    serving: it has no gradient.  quantize_q8 and rms_norm_q8 begin every row at a
    multiple of 16 bytes; with rows that do not a call takes up to 2.6 times as
    long."""
    if torch.is_grad_enabled():
        _no_graph(x.scale, w.scale, bias, out)
    if x.group or w.group:
        raise ValueError("a product takes one scale a row (group 0)")
    rows, width, xs = _q8(x, "x")
    n, length, wst = _q8(w, "w")
    dev = x.q.device
    if length != width or w.q.device != dev:
        raise ValueError("w must have x's width and device")
    if bias is not None:
        _vec1(bias, "bias", n, torch.float32, dev)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if out is None:
        y, ys = _empty(stream, (rows, n), dtype, dev), n
    else:
        y, ys = out, _rows(out, "out")
        if out.shape != (rows, n) or out.dtype != dtype or out.device != dev:
            raise ValueError("out must match the product's shape and device and the type asked for")
    o = Int8Opts(rows, width, n, _DTYPES[dtype], 0)
    _run("sgc_int8_linear", dev, stream, C.byref(o), x.q.data_ptr(), xs, x.scale.data_ptr(), w.q.data_ptr(), wst,
         w.scale.data_ptr(), _ptr(bias), y.data_ptr(), ys)
    if out is not None:
        _written(out)
    return y
