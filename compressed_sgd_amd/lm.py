"""The loss end of a language model: layer norm, token log probabilities and
distillation from a teacher's top entries, each with its gradient.

Thin marshalling over the C ABI (include/sgc.h), like the rest of the
binding; the calls are re-exported by the package.  Rows are taken from 2-D
tensors whose last dimension is contiguous; any row stride is allowed.  The
gradients are explicit calls (no autograd): what the backward calls need is
in the forward calls' results.  A tensor that requires grad is refused while
grad mode is on, since its gradient would be lost in silence: call under
torch.no_grad(), from an autograd.Function, or with detached tensors.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass
from typing import Optional

import torch

from . import SGCError, _check, _on, lib, workspace

F32, BF16, F16 = 0, 1, 2
NORM_ADD_GRADS = 1
TOKEN_I32, TOKEN_I64 = 0, 1
TOP_MAX = 256
LM_WS_NONE = 1
DISTILL_RENORM, DISTILL_TAIL = 0, 1

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


class NormOpts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("dtype", C.c_int32), ("wdtype", C.c_int32),
                ("eps", C.c_float), ("flags", C.c_int32)]


class LogprobOpts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("vocab", C.c_int64), ("dtype", C.c_int32), ("token_type", C.c_int32),
                ("top", C.c_int32), ("scale", C.c_float)]


class DistillOpts(C.Structure):
    _fields_ = [("rows", C.c_int64), ("vocab", C.c_int64), ("dtype", C.c_int32), ("top", C.c_int32),
                ("mode", C.c_int32), ("scale", C.c_float), ("teacher_scale", C.c_float), ("reserved", C.c_int32)]


def _declare(L) -> None:
    P, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
    for name, args, res in (
            ("sgc_layer_norm", [P, P, i64, P, P, P, i64, P, P, P], C.c_int),
            ("sgc_layer_norm_backward_workspace", [P], sz),
            ("sgc_layer_norm_backward", [P, P, i64, P, i64, P, P, P, P, i64, P, P, P, sz, P], C.c_int),
            ("sgc_token_logprobs_workspace", [P], sz),
            ("sgc_token_logprobs", [P, P, i64, P, P, P, P, P, P, P, P, sz, P], C.c_int),
            ("sgc_token_logprobs_backward", [P, P, i64, P, P, P, P, P, P, i64, P], C.c_int),
            ("sgc_distill_workspace", [P], sz),
            ("sgc_distill", [P, P, i64, P, P, P, P, P, P, i64, P, P, sz, P], C.c_int),
            ("sgc_distill_backward", [P, P, i64, P, P, P, P, P, i64, P], C.c_int)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


def _empty(stream, shape, dtype, device) -> torch.Tensor:
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with _on(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device, stream) -> int:
    """The handle of the call's stream (the current one's without the Stream object around it)."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _no_graph(*tensors: Optional[torch.Tensor]) -> None:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("this call records no graph: call it under torch.no_grad() or with detached tensors")


def _written(*tensors: Optional[torch.Tensor]) -> None:
    """Tells autograd that the caller's buffers hold other values now."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _rows(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None) -> int:
    """Checks a 2-D device tensor of rows; its row stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if t.dim() != 2 or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be 2-D float32, bfloat16 or float16")
    stride = t.stride()
    if stride[1] != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must match the input's shape, type and device")
    return stride[0]


def _vec(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> None:
    """Checks a contiguous operand of a known shape, type and device (None passes)."""
    if t is not None and (t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _vec1(t: Optional[torch.Tensor], name: str, n: int, dtype, device) -> None:
    """_vec for one dimension of n elements."""
    if t is not None and (t.numel() != n or t.dim() != 1 or t.dtype != dtype or t.device != device
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape ({n},) on {device}")


def _status(t: Optional[torch.Tensor], device) -> None:
    _vec1(t, "status", 1, torch.int32, device)


def _scratch(need: int, ws: Optional[torch.Tensor], device, slot: str, stream, what: str) -> Optional[torch.Tensor]:
    if need == 0:
        raise SGCError(-1, what)
    if ws is not None and (ws.device != device or not ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    if need == LM_WS_NONE or ws is not None:
        return ws
    return workspace(need, device, slot, stream)


# --------------------------------------------------------------- layer norm
@dataclass
class Normalized:
    y: torch.Tensor
    mean: torch.Tensor   # float32 [rows]
    rstd: torch.Tensor   # float32 [rows]


@dataclass
class NormGrads:
    dx: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]   # float32 [cols]
    dbias: Optional[torch.Tensor]     # float32 [cols]


def _affine(weight, bias, x, cols, dev) -> int:
    wdt = weight.dtype if weight is not None else bias.dtype if bias is not None else torch.float32
    if wdt != torch.float32 and wdt != x.dtype:
        raise ValueError("weight and bias must be float32 or the type of x")
    _vec1(weight, "weight", cols, wdt, dev)
    _vec1(bias, "bias", cols, wdt, dev)
    return _DTYPES[wdt]


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None, stream=None) -> Normalized:
    """Layer norm of every row of x [rows, cols]; out may be x."""
    _no_graph(x, weight, bias, out)
    xs = _rows(x, "x")
    rows, cols = x.shape
    dev = x.device
    wdt = _affine(weight, bias, x, cols, dev)
    if out is None:
        y, ys = _empty(stream, (rows, cols), x.dtype, dev), cols
    else:
        y, ys = out, _rows(out, "out", x)
    mean = _empty(stream, (rows,), torch.float32, dev)
    rstd = _empty(stream, (rows,), torch.float32, dev)
    o = NormOpts(rows, cols, _DTYPES[x.dtype], wdt, eps, 0)
    _check(lib().sgc_layer_norm(C.byref(o), _ptr(x), xs, _ptr(weight), _ptr(bias), _ptr(y), ys, _ptr(mean),
                                _ptr(rstd), _stream(dev, stream)), "sgc_layer_norm")
    _written(out)
    return Normalized(y, mean, rstd)


def layer_norm_backward_workspace_bytes(rows: int, cols: int, dtype: torch.dtype = torch.float32) -> int:
    return int(lib().sgc_layer_norm_backward_workspace(C.byref(NormOpts(rows, cols, _DTYPES[dtype], F32, 0.0, 0))))


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                        rstd: torch.Tensor, *, dx: Optional[torch.Tensor] = None,
                        dweight: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                        accumulate: bool = False, want_dx: bool = True, ws: Optional[torch.Tensor] = None,
                        stream=None) -> NormGrads:
    """Gradients of layer_norm.  dweight and dbias (float32, e.g. slices of a
    flat gradient) are written, or with accumulate added to; new ones are made
    where none is given.  dx may be dy or x."""
    _no_graph(dy, x, weight, mean, rstd, dx, dweight, dbias)
    xs = _rows(x, "x")
    dys = _rows(dy, "dy", x)
    rows, cols = x.shape
    dev = x.device
    wdt = _affine(weight, None, x, cols, dev)
    for t, name, n in ((mean, "mean", rows), (rstd, "rstd", rows), (dweight, "dweight", cols),
                       (dbias, "dbias", cols)):
        _vec1(t, name, n, torch.float32, dev)
    if accumulate and (dweight is None or dbias is None):
        raise ValueError("accumulate needs dweight and dbias")
    given = (dx, dweight, dbias)
    if dx is None and want_dx:
        dx = _empty(stream, (rows, cols), x.dtype, dev)
    dxs = _rows(dx, "dx", x) if dx is not None else 0
    if dweight is None:
        dweight = _empty(stream, (cols,), torch.float32, dev)
    if dbias is None:
        dbias = _empty(stream, (cols,), torch.float32, dev)
    o = NormOpts(rows, cols, _DTYPES[x.dtype], wdt, 0.0, NORM_ADD_GRADS if accumulate else 0)
    L = lib()
    need = L.sgc_layer_norm_backward_workspace(C.byref(o))
    ws = _scratch(need, ws, dev, "layer_norm", stream, "sgc_layer_norm_backward_workspace")
    _check(L.sgc_layer_norm_backward(C.byref(o), _ptr(dy), dys, _ptr(x), xs, _ptr(weight), _ptr(mean), _ptr(rstd),
                                     _ptr(dx), dxs, _ptr(dweight), _ptr(dbias), _ptr(ws),
                                     0 if ws is None else ws.numel(), _stream(dev, stream)),
           "sgc_layer_norm_backward")
    _written(*given)
    return NormGrads(dx, dweight, dbias)


# ------------------------------------------------------- token log probabilities
@dataclass
class TokenLogprobs:
    logp: Optional[torch.Tensor]      # float32 [rows]; None without tokens
    entropy: torch.Tensor             # float32 [rows]
    stats: torch.Tensor               # float32 [rows, 2]: the row's maximum and sum, for the backward call
    top_idx: Optional[torch.Tensor]   # int32 [rows, top], best first
    top_logp: Optional[torch.Tensor]  # float32 [rows, top]


def _tokens(tokens: Optional[torch.Tensor], rows: int, device) -> int:
    if tokens is None:
        return TOKEN_I64
    dt = tokens.dtype
    if dt != torch.int64 and dt != torch.int32:
        raise ValueError("tokens must be int32 or int64")
    _vec1(tokens, "tokens", rows, dt, device)
    return TOKEN_I64 if dt == torch.int64 else TOKEN_I32


def token_logprobs_workspace_bytes(rows: int, vocab: int, *, top: int = 0, dtype: torch.dtype = torch.float32) -> int:
    """Workspace bytes of one token_logprobs call (1: it needs none)."""
    return int(lib().sgc_token_logprobs_workspace(C.byref(LogprobOpts(rows, vocab, _DTYPES[dtype], TOKEN_I64, top,
                                                                      1.0))))


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, scale: float = 1.0, top: int = 0,
                   out: Optional[TokenLogprobs] = None, status: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, stream=None) -> TokenLogprobs:
    """Log probability of tokens [rows] under softmax(scale * logits) [rows,
    vocab], the entropy, and the `top` likeliest tokens of every row.

    A negative token is none (logp 0).  status (int32 [1]) collects
    STATUS_BAD_INPUT for a token past the vocabulary, whose logp is NaN.
    """
    _no_graph(logits)
    zs = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    tt = _tokens(tokens, rows, dev)
    _status(status, dev)
    f32 = torch.float32
    given = out
    if out is None:
        out = TokenLogprobs(None if tokens is None else _empty(stream, (rows,), f32, dev),
                            _empty(stream, (rows,), f32, dev), _empty(stream, (rows, 2), f32, dev),
                            _empty(stream, (rows, top), torch.int32, dev) if top > 0 else None,
                            _empty(stream, (rows, top), f32, dev) if top > 0 else None)
    else:
        for t, name, shape, dt in ((out.logp, "out.logp", (rows,), f32), (out.entropy, "out.entropy", (rows,), f32),
                                   (out.stats, "out.stats", (rows, 2), f32),
                                   (out.top_idx, "out.top_idx", (rows, top), torch.int32),
                                   (out.top_logp, "out.top_logp", (rows, top), f32)):
            _vec(t, name, shape, dt, dev)
    o = LogprobOpts(rows, vocab, _DTYPES[logits.dtype], tt, top, scale)
    L = lib()
    need = L.sgc_token_logprobs_workspace(C.byref(o))
    ws = _scratch(need, ws, dev, "token_logprobs", stream, "sgc_token_logprobs")
    _check(L.sgc_token_logprobs(C.byref(o), _ptr(logits), zs, _ptr(tokens), _ptr(out.logp), _ptr(out.entropy),
                                _ptr(out.stats), _ptr(out.top_idx), _ptr(out.top_logp), _ptr(status), _ptr(ws),
                                0 if ws is None else ws.numel(), _stream(dev, stream)), "sgc_token_logprobs")
    if given is not None:
        _written(out.logp, out.entropy, out.stats, out.top_idx, out.top_logp)
    return out


def token_logprobs_backward(logits: torch.Tensor, tokens: Optional[torch.Tensor], stats: torch.Tensor,
                            entropy: Optional[torch.Tensor], dlogp: Optional[torch.Tensor],
                            dentropy: Optional[torch.Tensor] = None, *, scale: float = 1.0,
                            dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits from those of logp and entropy (either may be
    None); stats and entropy are the forward call's.  dlogits may be logits."""
    _no_graph(logits, stats, entropy, dlogp, dentropy, dlogits)
    zs = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    tt = _tokens(tokens, rows, dev)
    f32 = torch.float32
    _vec(stats, "stats", (rows, 2), f32, dev)
    for t, name in ((entropy, "entropy"), (dlogp, "dlogp"), (dentropy, "dentropy")):
        _vec1(t, name, rows, f32, dev)
    ds, given = vocab, dlogits
    if dlogits is None:
        dlogits = _empty(stream, (rows, vocab), logits.dtype, dev)
    else:
        ds = _rows(dlogits, "dlogits", logits)
    o = LogprobOpts(rows, vocab, _DTYPES[logits.dtype], tt, 0, scale)
    _check(lib().sgc_token_logprobs_backward(C.byref(o), _ptr(logits), zs, _ptr(tokens), _ptr(stats), _ptr(entropy),
                                             _ptr(dlogp), _ptr(dentropy), _ptr(dlogits), ds, _stream(dev, stream)),
           "sgc_token_logprobs_backward")
    _written(given)
    return dlogits


# ------------------------------------------------------------ distillation
@dataclass
class Distilled:
    loss: torch.Tensor                # float32 [rows]
    stats: torch.Tensor               # float32 [rows, 4], for the backward call
    dlogits: Optional[torch.Tensor]


def _entries(t_idx: torch.Tensor, t_val: torch.Tensor, rows: int, device) -> int:
    if t_idx.dim() != 2:
        raise ValueError("t_idx must be 2-D [rows, top]")
    shape = (rows, t_idx.shape[1])
    _vec(t_idx, "t_idx", shape, torch.int32, device)
    _vec(t_val, "t_val", shape, torch.float32, device)
    return shape[1]


def distill_workspace_bytes(rows: int, vocab: int, top: int, *, dtype: torch.dtype = torch.float32) -> int:
    """Workspace bytes of one distill call (1: it needs none)."""
    return int(lib().sgc_distill_workspace(C.byref(DistillOpts(rows, vocab, _DTYPES[dtype], top, DISTILL_RENORM, 1.0,
                                                               1.0, 0))))


def distill(logits: torch.Tensor, t_idx: torch.Tensor, t_val: torch.Tensor, *, mode: int = DISTILL_RENORM,
            scale: float = 1.0, teacher_scale: float = 1.0, dloss: Optional[torch.Tensor] = None,
            dlogits: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None, stream=None) -> Distilled:
    """Divergence of softmax(scale * logits) from a teacher's top entries.

    With dloss [rows] (the rows' upstream gradients) or a dlogits buffer the
    gradient comes in the same call; dlogits may be logits.  status (int32
    [1]) collects STATUS_CORRUPT for a row with a bad or repeated index.
    """
    _no_graph(logits, t_val, dloss, dlogits)
    zs = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    top = _entries(t_idx, t_val, rows, dev)
    _status(status, dev)
    _vec1(dloss, "dloss", rows, torch.float32, dev)
    ds, given = vocab, dlogits
    if dlogits is not None:
        ds = _rows(dlogits, "dlogits", logits)
    elif dloss is not None:
        dlogits = _empty(stream, (rows, vocab), logits.dtype, dev)
    loss = _empty(stream, (rows,), torch.float32, dev)
    stats = _empty(stream, (rows, 4), torch.float32, dev)
    o = DistillOpts(rows, vocab, _DTYPES[logits.dtype], top, mode, scale, teacher_scale, 0)
    L = lib()
    need = L.sgc_distill_workspace(C.byref(o))
    ws = _scratch(need, ws, dev, "distill", stream, "sgc_distill")
    _check(L.sgc_distill(C.byref(o), _ptr(logits), zs, _ptr(t_idx), _ptr(t_val), _ptr(loss), _ptr(stats),
                         _ptr(dloss), _ptr(dlogits), ds, _ptr(status), _ptr(ws), 0 if ws is None else ws.numel(),
                         _stream(dev, stream)), "sgc_distill")
    _written(given)
    return Distilled(loss, stats, dlogits)


def distill_backward(logits: torch.Tensor, t_idx: torch.Tensor, t_val: torch.Tensor, stats: torch.Tensor,
                     dloss: Optional[torch.Tensor] = None, *, mode: int = DISTILL_RENORM, scale: float = 1.0,
                     teacher_scale: float = 1.0, dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits from the rows' upstream gradients (None: 1) and
    the loss call's stats.  dlogits may be logits."""
    _no_graph(logits, t_val, stats, dloss, dlogits)
    zs = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev = logits.device
    top = _entries(t_idx, t_val, rows, dev)
    _vec(stats, "stats", (rows, 4), torch.float32, dev)
    _vec1(dloss, "dloss", rows, torch.float32, dev)
    ds, given = vocab, dlogits
    if dlogits is None:
        dlogits = _empty(stream, (rows, vocab), logits.dtype, dev)
    else:
        ds = _rows(dlogits, "dlogits", logits)
    o = DistillOpts(rows, vocab, _DTYPES[logits.dtype], top, mode, scale, teacher_scale, 0)
    _check(lib().sgc_distill_backward(C.byref(o), _ptr(logits), zs, _ptr(t_idx), _ptr(t_val), _ptr(stats),
                                      _ptr(dloss), _ptr(dlogits), ds, _stream(dev, stream)), "sgc_distill_backward")
    _written(given)
    return dlogits
