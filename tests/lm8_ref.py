"""Plain forms of the 8-bit operators and of RMS norm: whole numbers by the
definition's own fp32 steps (bit for bit), the rest in 64 bits, with how far an
fp32 computation may be from it.

U is half a step of fp32 relative to the value.  A sum over a row is at most
`depth` additions deep, so its error is at most depth * U times the sum of its
terms' magnitudes.
"""
from __future__ import annotations

import torch

import lm_ref
from lm_ref import U, dbl


def depth(n):
    """Rows up to 16384 stay in registers: 16 elements a thread, 10 steps across threads; longer ones go by
    strides of 1024 threads."""
    return 32 + n // 1024


# ------------------------------------------------------------------ 8 bits
def quantize(x, group):
    """q (int8) and scale (fp32) of x, every operation rounded to fp32 as the definition says."""
    rows, cols = x.shape
    width = group or cols
    x = x.detach().cpu().float()
    q, scale = torch.zeros(rows, cols, dtype=torch.int8), []
    for a in range(0, cols, width):
        p = x[:, a:a + width]
        top = p.abs().amax(1, keepdim=True)  # NaN where there is one
        small = top < 2.0 ** -100
        pre = torch.where(small, 2.0 ** 100, 1.0)
        r = torch.full_like(top, 127.0) / (top * pre)
        v = torch.round((p * pre) * r)
        fine = torch.isfinite(top)
        q[:, a:a + width] = torch.where(fine & (top > 0), v, 0.0).to(torch.int8)
        scale.append(torch.where(fine, top / torch.full_like(top, 127.0), float("nan")))
    return q, torch.cat(scale, 1)


def values(q, scale, group):
    """q * scale, rounded to fp32."""
    q, scale = q.cpu(), scale.cpu()
    if group:
        scale = scale.repeat_interleave(group, dim=1)[:, :q.shape[1]]
    return q.float() * scale


# ---------------------------------------------------------------- RMS norm
def stream(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def rms(s, w, eps):
    """y, rstd and how far they may be."""
    s = dbl(s)
    n = s.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else dbl(w)
    ms = (s * s).mean(1)
    rstd = (ms + eps) ** -0.5
    t_rstd = rstd * (0.5 * (depth(n) + 3) * U * ms / (ms + eps) + 4 * U)
    y = s * rstd[:, None] * w
    t_y = (s * w).abs() * t_rstd[:, None] + 3 * U * y.abs()
    return (y, rstd), (t_y, t_rstd)


def rms_q8(s, w, eps):
    """q, scale, rstd and how far scale and rstd may be."""
    p = s.detach().cpu().float() * (torch.ones(s.shape[1]) if w is None else w.detach().cpu().float())
    q, sc = quantize(p, 0)
    (_, rstd), (_, t_rstd) = rms(s, w, eps)
    scale = sc.double() * rstd[:, None]
    return q, (scale, rstd), (sc.double() * t_rstd[:, None] + 2 * U * scale.abs(), t_rstd)


def backward(dy, x, w, mean, rstd, dsum):
    """dx, dweight, dbias for the given mean (None: RMS norm) and rstd, and how far they may be."""
    if mean is not None:
        (dx, dw, db), (t_dx, t_dw, t_db) = lm_ref.norm_backward(dy, x, w, mean, rstd)
    else:
        dy, x, rs = dbl(dy), dbl(x), dbl(rstd)[:, None]
        rows, n = x.shape
        w = torch.ones(n, dtype=torch.float64) if w is None else dbl(w)
        h, v = x * rs, dy * w
        c2 = (v * h).mean(1, keepdim=True)
        dx = rs * (v - h * c2)
        t_c2 = (depth(n) + 4) * U * (v * h).abs().mean(1, keepdim=True)
        t_dx = rs * (h.abs() * t_c2 + 4 * U * (v.abs() + 2 * (h * c2).abs()))
        dw, db = (dy * h).sum(0), None
        # the rows of a part one after the other, then the parts
        t_dw, t_db = (64 + rows // 64 + 2) * U * (dy * h).abs().sum(0), None
    if dsum is not None:
        dx = dx + dbl(dsum)
        t_dx = t_dx + U * dx.abs()
    return (dx, dw, db), (t_dx, t_dw, t_db)


def normed(x, w, b, mean, rstd):
    """x's normed rows for the given mean (None: RMS norm) and rstd, and how far they may be."""
    x, rs = dbl(x), dbl(rstd)[:, None]
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else dbl(w)
    b = torch.zeros(n, dtype=torch.float64) if b is None else dbl(b)
    m = torch.zeros_like(rs) if mean is None else dbl(mean)[:, None]
    h = (x - m) * rs
    t_h = U * (x.abs() + m.abs()) * rs + 2 * U * h.abs()
    y = h * w + b
    return y, t_h * w.abs() + 2 * U * (h * w).abs() + U * y.abs()


# ---------------------------------------------------------------- products
def product(xq, xscale, wq, wscale, bias):
    """y and how far it may be: the sum is exact, one rounding of it, one a scale, one of the bias' addition."""
    acc = dbl(xq) @ dbl(wq).t()
    y = acc * dbl(xscale) * dbl(wscale).t()
    t = 4 * U * y.abs()
    if bias is not None:
        y = y + dbl(bias)
        t = t + U * (y.abs() + t)
    return y, t
