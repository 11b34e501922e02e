"""Plain 64-bit forms of the language-model operators, from their formulas,
and how far an fp32 computation may be from them.

U is half a step of fp32 relative to the value.  A sum in any layout the
kernels use is at most DEPTH additions deep, so its error is at most DEPTH * U
times the sum of its terms' magnitudes; an exponential of y has the relative
error of y's own rounding, |y| * U for each operation on it, and a few U.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
DEPTH = 64
# powers of two below fp32's normal range are 0 in the kernels
FLUSH = 2.0 ** -126


def half_step(dtype, ref):
    """Rounding once to dtype: half a step of the value, or of the smallest one."""
    f = torch.finfo(dtype)
    return f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2


def dbl(t):
    return t.detach().cpu().double()


# --------------------------------------------------------------- layer norm
def norm(x, w, b, eps):
    """y, mean, rstd and how far y, mean and rstd may be."""
    x = dbl(x)
    n = x.shape[1]
    mean = x.mean(1)
    d = x - mean[:, None]
    var = (d * d).mean(1)
    rstd = (var + eps) ** -0.5
    w = torch.ones(n, dtype=torch.float64) if w is None else dbl(w)
    b = torch.zeros(n, dtype=torch.float64) if b is None else dbl(b)
    h = d * rstd[:, None]
    y = h * w + b
    t_mean = (DEPTH + 2) * U * x.abs().mean(1)
    # the variance: rounding of the sum, and the mean's error through every d
    t_var = (DEPTH + 4) * U * var + 2 * t_mean * d.abs().mean(1) + t_mean ** 2 + \
        2 * U * (x.abs() * d.abs()).mean(1)
    t_rstd = rstd * (0.5 * t_var / (var + eps) + 4 * U)
    t_h = (t_mean[:, None] + U * (x.abs() + mean.abs()[:, None])) * rstd[:, None] + \
        d.abs() * t_rstd[:, None] + 2 * U * h.abs()
    t_y = t_h * w.abs() + 2 * U * (h * w).abs() + 2 * U * y.abs()
    return (y, mean, rstd), (t_y, t_mean + U * mean.abs(), t_rstd)


def norm_backward(dy, x, w, mean, rstd):
    """dx, dweight, dbias for the given mean and rstd, and how far they may be."""
    dy, x, mean, rstd = dbl(dy), dbl(x), dbl(mean)[:, None], dbl(rstd)[:, None]
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else dbl(w)
    h = (x - mean) * rstd
    t_h = 2 * U * (x.abs() + mean.abs()) * rstd + U * h.abs()
    v = dy * w
    c1, c2 = v.mean(1, keepdim=True), (v * h).mean(1, keepdim=True)
    dx = rstd * (v - c1 - h * c2)
    t_c1 = (DEPTH + 3) * U * v.abs().mean(1, keepdim=True)
    t_c2 = (DEPTH + 4) * U * (v * h).abs().mean(1, keepdim=True) + (v.abs() * t_h).mean(1, keepdim=True)
    t_dx = rstd * (t_c1 + h.abs() * t_c2 + t_h * c2.abs() + 4 * U * (v.abs() + c1.abs() + (h * c2).abs()))
    rows = x.shape[0]
    deep = DEPTH + min(rows, 512)  # rows of a part one after the other, then the parts
    dw, db = (dy * h).sum(0), dy.sum(0)
    t_dw = (deep + 2) * U * (dy * h).abs().sum(0) + (dy.abs() * t_h).sum(0)
    t_db = deep * U * dy.abs().sum(0)
    return (dx, dw, db), (t_dx, t_dw, t_db)


# ------------------------------------------------------- token log probabilities
class Softmax:
    """log p of scale * z for every row; rows of -inf alone have none, rows
    with NaN or +inf are NaN."""

    def __init__(self, z, scale):
        z = dbl(z)
        self.scale = scale
        self.none = (z == -float("inf")).all(1)
        self.nan = torch.isnan(z).any(1) | (z == float("inf")).any(1)
        m = z.amax(1, keepdim=True)
        m = torch.where(self.none[:, None] | ~torch.isfinite(m), 0.0, m)
        self.y = (z - m) * scale
        e = self.y.exp()
        s = e.sum(1, keepdim=True)
        self.log_s = s.log()
        self.lp = self.y - self.log_s
        self.lp[self.none] = -float("inf")
        self.lp[self.nan] = float("nan")
        self.p = torch.where(self.none[:, None], 0.0, self.lp.exp())
        pl = torch.where(self.p == 0, 0.0, self.p * self.lp)
        self.H = -pl.sum(1)
        yc = self.y.clamp(min=-1e4)
        py = torch.where(self.p == 0, 0.0, self.p * yc)
        self.mean_y = py.abs().sum(1, keepdim=True)
        self.mean_yy = (py * yc).abs().sum(1, keepdim=True)
        ls = torch.where(self.none[:, None], 0.0, self.log_s)
        # ln s: the sum's depth, the exponents' rounding, the logarithm's
        self.t_ls = U * (DEPTH + 4 + 4 * self.mean_y + 2 * ls.abs())
        ya = torch.where(torch.isfinite(self.y), self.y.abs(), 0.0)
        self.t_lp = self.t_ls + U * (4 * ya + 2 * ls.abs())
        self.t_H = self.t_ls + U * ((DEPTH + 8) * self.mean_y + 4 * self.mean_yy + 2 * ls.abs())


def logprobs(z, tokens, scale, top):
    """logp, entropy, top_idx, top_logp and the tolerances of logp, entropy, top_logp."""
    sm = Softmax(z, scale)
    V = z.shape[1]
    logp = t_logp = None
    if tokens is not None:
        tok = tokens.cpu().long()
        at = tok.clamp(0, V - 1)[:, None]
        logp = sm.lp.gather(1, at)[:, 0]
        logp = torch.where(tok < 0, 0.0, torch.where(tok >= V, float("nan"), logp))
        t_logp = sm.t_lp.gather(1, at)[:, 0]
    # order: NaN, +inf, ..., -inf; equal values by the lower place
    key = dbl(z) + 0.0
    order = sorted_places(key, top)
    top_logp = sm.lp.gather(1, order)
    return sm, (logp, sm.H, order, top_logp), (t_logp, sm.t_H[:, 0], sm.t_lp.gather(1, order))


def sorted_places(key, top):
    nan = torch.isnan(key)
    key = torch.where(nan, 0.0, key)
    by_value = torch.sort(key, dim=1, descending=True, stable=True).indices
    first = torch.sort(nan.gather(1, by_value).to(torch.int8), dim=1, descending=True, stable=True).indices
    return by_value.gather(1, first)[:, :top]


def logprobs_backward(sm, tokens, g, h):
    """dlogits, and how far an fp32 computation of it may be (before rounding to its type)."""
    rows, V = sm.lp.shape
    g = torch.zeros(rows, dtype=torch.float64) if g is None else dbl(g)
    h = torch.zeros(rows, dtype=torch.float64) if h is None else dbl(h)
    hot = torch.zeros(rows, V, dtype=torch.float64)
    if tokens is not None:
        tok = tokens.cpu().long()
        ok = (tok >= 0) & (tok < V)
        g = torch.where(ok, g, 0.0)
        hot[torch.arange(rows)[ok], tok[ok]] = 1.0
    g, h = g[:, None], h[:, None]
    lp = torch.where(sm.p == 0, 0.0, sm.lp)
    H = sm.H[:, None]
    d = sm.scale * (g * (hot - sm.p) - h * sm.p * (lp + H))
    tol = sm.scale * (g.abs() * (sm.p * (sm.t_lp + 4 * U) + 2 * U * hot) + h.abs() * sm.p * (
        (lp + H).abs() * (sm.t_lp + 4 * U) + sm.t_lp + sm.t_H + 4 * U * (lp.abs() + H.abs()))) + 4 * U * d.abs()
    tol = tol + sm.scale * (g.abs() + h.abs() * (lp + H).abs()) * FLUSH
    zero = sm.none | ((g == 0) & (h == 0))[:, 0]
    d[zero] = 0.0
    tol[zero] = 0.0
    return d, tol


# ------------------------------------------------------------ distillation
def teacher(t_idx, t_val, vocab, tail, teacher_scale=1.0):
    """t, log t, u of every row, rows that are bad, rows without an entry, tolerance of log t and u."""
    idx = t_idx.cpu().long()
    v = dbl(t_val) * teacher_scale
    v = torch.where(idx < 0, -float("inf"), v)
    bad = (idx < -1).any(1) | (idx >= vocab).any(1)
    srt = idx.sort(1).values
    bad |= ((srt[:, 1:] == srt[:, :-1]) & (srt[:, 1:] >= 0)).any(1)
    if tail:
        lt, t_lt = v, U * (4 + 4 * v.abs())
    else:
        m = v.amax(1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, 0.0)
        ls = (v - m).exp().sum(1, keepdim=True).log()
        lt = torch.where(v == -float("inf"), v, v - m - ls)
        t_lt = U * (DEPTH + 8 + 8 * (v - m).abs() + 4 * ls.abs())
    t_lt = torch.where(torch.isfinite(lt), t_lt, 0.0)
    t = lt.exp()
    total = t.sum(1, keepdim=True)
    u = (1.0 - total).clamp(min=0.0) if tail else torch.zeros_like(total)
    t_u = (DEPTH + 2) * U * total + (t * t_lt).sum(1, keepdim=True) if tail else torch.zeros_like(total)
    if not tail:
        total = torch.where(total > 0, torch.ones_like(total), total)
    return dict(idx=idx, t=t, lt=lt, u=u, total=total, bad=bad, t_lt=t_lt, t_u=t_u)


def distill(z, t_idx, t_val, tail, scale, teacher_scale=1.0, g=None):
    """loss, dlogits and their tolerances (dlogits' before rounding to its type)."""
    rows, V = z.shape
    sm = Softmax(z, scale)
    te = teacher(t_idx, t_val, V, tail, teacher_scale)
    idx, t, lt, u = te["idx"], te["t"], te["lt"], te["u"]
    at = idx.clamp(0, V - 1)
    has = (idx >= 0) & (idx < V)
    inside = torch.zeros(rows, V + 1, dtype=torch.bool)
    inside.scatter_(1, torch.where(has, at, V), True)
    inside = inside[:, :V]
    outside = torch.where(inside, 0.0, sm.p).sum(1, keepdim=True)
    lq = sm.lp.gather(1, at)
    live = has & (t != 0)
    term = torch.where(live, t * (lt - lq), 0.0)
    tl = torch.where(live, t * (te["t_lt"] * (1 + (lt - lq).abs()) + sm.t_lp.gather(1, at)
                                + DEPTH * U * (lt.abs() + lq.abs())), 0.0).sum(1)
    loss = term.sum(1)
    tail_on = (u > 0) & (outside > 0)
    lu, lo = u.clamp(min=1e-300).log(), outside.clamp(min=1e-300).log()
    loss = loss + torch.where(tail_on, u * (lu - lo), 0.0)[:, 0]
    t_tail = te["t_u"] * (1 + (lu - lo).abs()) + u * (2 * sm.t_ls + U * (DEPTH + 4 * (lu.abs() + lo.abs()))
                                                      + 4 * U * (sm.y.clamp(min=-90.0).abs().amax(1, keepdim=True)))
    # where the exact rest is smaller than its own error the kernel may find none
    tl = tl + torch.where(tail_on | (te["t_u"] > 0), t_tail, 0.0)[:, 0]
    skip = te["bad"] | sm.none
    if not tail:
        skip = skip | (te["total"] == 0)[:, 0]
    loss = torch.where(skip, 0.0, loss)
    loss = torch.where(te["bad"], float("nan"), loss)
    g = torch.ones(rows, dtype=torch.float64) if g is None else dbl(g)
    gs = (g * scale)[:, None]
    mass = te["total"] + u
    share = torch.where(tail_on & ~inside, sm.p / outside.clamp(min=1e-300), 0.0)
    tt = torch.zeros(rows, V + 1, dtype=torch.float64).scatter_(1, torch.where(has, at, V), t)[:, :V]
    t_tt = torch.zeros(rows, V + 1, dtype=torch.float64).scatter_(
        1, torch.where(has, at, V), t * (te["t_lt"] + 4 * U))[:, :V]
    d = gs * (mass * sm.p - tt - u * share)
    tol = gs.abs() * (mass * sm.p * (sm.t_lp + 6 * U) + t_tt + te["t_u"] * (sm.p + share)
                      + u * share * (2 * sm.t_lp + (DEPTH + 8) * U)) + 4 * U * d.abs()
    tol = tol + gs.abs() * FLUSH * (mass + torch.where(tail_on, u / outside.clamp(min=1e-300), 0.0))
    zero = skip | (g == 0)
    d[zero] = 0.0
    tol[zero] = 0.0
    return loss, d, tl + U * loss.abs(), tol


# ------------------------------------------------------------------ compare
def close(got, ref, tol, what, dtype=None):
    """got within tol (plus one rounding to dtype) of ref; infinities and NaN alike."""
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)} != {tuple(ref.shape)}"
    t = tol if dtype is None else tol + half_step(dtype, ref)
    # past the largest finite value, rounding gives infinity
    f = torch.finfo(got.dtype)
    ref = torch.where(ref.abs() >= f.max * (1 + f.eps / 4), ref.sign() * float("inf"), ref)
    nan = torch.isnan(ref)
    inf = torch.isinf(ref)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN at other places"
    assert torch.equal(g[inf], ref[inf]), f"{what}: infinities differ"
    fine = ~(nan | inf)
    off = (g - ref).abs()[fine] - t.expand_as(ref)[fine]
    if off.numel() and float(off.max()) > 0:
        k = int(off.argmax())
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {off.numel()} too far, worst got "
                             f"{float(g[fine][k])!r} want {float(ref[fine][k])!r} tolerance "
                             f"{float(t.expand_as(ref)[fine][k]):.3g}")
