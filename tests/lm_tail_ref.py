"""Distillation with the tail in 64 bits from sums in the log domain, so that
the mass outside a teacher's list is right however small it is, and how far an
fp32 computation may be from it.

U is half a step of fp32.  DEPTH bounds the chain of additions of any sum here:
at most 512 elements of a row go to one thread, in two chains, and the joins
add 16.  The hardware's exponential gives 0 below 2^-126 (FLUSH) of the largest
term of the sum it belongs to.
"""
from __future__ import annotations

import math

import torch

import lm_ref
from lm_ref import FLUSH, U, dbl

DEPTH = 512 // 2 + 16
INF = float("inf")
# a mass outside the list that lies this many powers of two below the row's
# maximum counts as none
GONE = 1074


def distill(z, t_idx, t_val, scale, g):
    """loss, dlogits, and how far each may be (dlogits before rounding to its
    type).  Every index is inside the vocabulary, every logit finite or -inf."""
    rows, V = z.shape
    z, g = dbl(z), dbl(g)
    te = lm_ref.teacher(t_idx, t_val, V, True)
    idx, t, lt, u, t_lt, t_u = (te[k] for k in ("idx", "t", "lt", "u", "t_lt", "t_u"))
    inside = torch.zeros(rows, V, dtype=torch.bool).scatter_(1, idx, True)
    m = z.amax(1, keepdim=True)
    zo = torch.where(inside, -INF, z)
    mo = zo.amax(1, keepdim=True)
    y = (z - m) * scale
    yo = torch.where(inside, -INF, (zo - mo) * scale)
    ls, lo = torch.logsumexp(y, 1, keepdim=True), torch.logsumexp(yo, 1, keepdim=True)
    D = (m - mo) * scale                                   # nats from the maximum to the outside's
    live = (u > 0) & (D / math.log(2.0) <= GONE)
    D = torch.where(live, D, 0.0)
    lp, l1q = y - ls, lo - D - ls                          # log q and log(1 - Q)
    p = lp.exp()
    share = torch.where(live & ~inside, (yo - lo).exp(), 0.0)
    lu = u.clamp(min=1e-300).log()
    lq = lp.gather(1, idx)
    term = torch.where(t > 0, t * (lt - lq), 0.0)
    loss = (term.sum(1, keepdim=True) + torch.where(live, u * (lu - l1q), 0.0))[:, 0]
    mass = t.sum(1, keepdim=True) + u
    tt = torch.zeros(rows, V, dtype=torch.float64).scatter_(1, idx, t)
    gs = (g * scale)[:, None]
    d = gs * (mass * p - tt - u * share)

    def t_log_sum(y, ls):
        # the depth of the sum, the exponents' rounding (4 operations on y), the logarithm
        mean = torch.where(y == -INF, 0.0, (y - ls).exp() * y.clamp(min=-1e4).abs()).sum(1, keepdim=True)
        return U * (DEPTH + 4 + 4 * mean + 2 * ls.abs())

    fin = lambda x: torch.where(torch.isfinite(x), x.abs(), 0.0)
    t_ls, t_lo = t_log_sum(y, ls), t_log_sum(yo, lo)
    t_lp = t_ls + U * (4 * fin(y) + 2 * ls.abs())
    t_l1q = t_lo + t_ls + U * (8 * D + 4 * (lo.abs() + ls.abs()))
    t_term = torch.where(t > 0, t * (t_lt * (1 + (lt - lq).abs()) + t_lp.gather(1, idx)
                                     + DEPTH * U * (lt.abs() + lq.abs())), 0.0).sum(1, keepdim=True)
    t_tail = torch.where(live, t_u * (1 + (lu - l1q).abs()) + u * (t_l1q + 4 * U * (lu.abs() + l1q.abs())), 0.0)
    t_loss = (t_term + t_tail)[:, 0] + U * loss.abs()
    # outside: either measured from the outside's maximum, or from the row's
    # with the distance taken back
    t_share = t_lo + U * (4 * (fin(yo) + D) + 8)
    t_tt = torch.zeros(rows, V, dtype=torch.float64).scatter_(1, idx, t * (t_lt + 4 * U))
    t_d = gs.abs() * (mass * p * (t_lp + 6 * U) + t_tt + t_u * (p + share) + u * share * t_share
                      + FLUSH * (mass + 2 * u)) + 4 * U * d.abs()
    d[g == 0], t_d[g == 0] = 0.0, 0.0
    return loss, d, t_loss, t_d
