"""Distillation with the tail where the student's mass lies on the teacher's
list: the outside measured from its own maximum, so that neither the loss nor
the gradient loses it or overflows, by every kernel that computes them.
"""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm_tail_ref
from gpu_util import announce
from lm_ref import close

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")
GAPS = [0.0, 9.0, 20.0, 23.0, 30.0, 60.0, 80.0, 84.0, 86.0, 87.0, 88.0, 89.0, 90.0, 110.0, 300.0, 700.0]


def far_rows(gaps, vocab, k, scale, dtype, seed):
    """Rows whose listed logits lie `gap` nats above all others, and their teacher's list."""
    g = torch.Generator().manual_seed(seed)
    rows = len(gaps)
    wide = torch.float64 if dtype == torch.float64 else torch.float32
    z = torch.randn(rows, vocab, generator=g, dtype=wide).clamp(-3, 3) / scale
    idx = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)])
    up = (torch.rand(rows, k, generator=g, dtype=wide) * 2 + 3 + torch.tensor(gaps, dtype=wide)[:, None]) / scale
    z.scatter_(1, idx, up)
    mass = torch.rand(rows, 1, generator=g) * 0.4 + 0.5
    val = torch.log_softmax(torch.randn(rows, k, generator=g), 1) + mass.log()
    return z.to(dtype), idx.int(), val


def check(z, idx, val, scale, g):
    loss, d, tl, td = lm_tail_ref.distill(z, idx, val, scale, g)
    kw = dict(mode=sgc.DISTILL_TAIL, scale=scale)
    zd, i, v, gd = z.cuda(), idx.cuda(), val.cuda(), g.cuda()
    one = sgc.distill(zd, i, v, **kw)
    close(one.loss, loss, tl, "loss")
    both = sgc.distill(zd, i, v, dloss=gd, **kw)
    close(both.loss, loss, tl, "loss of the call with the gradient")
    close(both.dlogits, d, td, "dlogits of the loss call", z.dtype)
    for s, what in ((one.stats, "loss call"), (both.stats, "call with the gradient")):
        close(sgc.distill_backward(zd, i, v, s, gd, **kw), d, td, f"dlogits from the stats of the {what}", z.dtype)
    return both


# (vocabulary, rows a gap): one wave, held rows of 4 to 16 waves, whole rows
# read twice, chunks of a row; many rows, by two waves; past the last-level cache
SHAPES = [(37, 1), (98, 1), (1003, 1), (2049, 1), (5003, 1), (5003, 40), (20011, 1), (40009, 1), (50001, 1),
          (60008, 1), (70001, 1), (131072, 1), (140001, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,repeat", SHAPES, ids=str)
def test_list_far_above_the_rest(vocab, repeat, dtype):
    scales = [0.25, 1.0, 4.0, 8.0] if vocab < 6000 else [1.0]
    for n, scale in enumerate(scales):
        gaps = GAPS * repeat
        announce(f"list far above the rest, {len(gaps)}x{vocab} {dtype} scale {scale}")
        z, idx, val = far_rows(gaps, vocab, 16, scale, dtype, vocab + n)
        g = torch.rand(len(gaps), generator=torch.Generator().manual_seed(n)) + 0.5
        g[1::3] = 65536.0                # a loss scale
        g[4::7] = 0.0
        check(z, idx, val, scale, g)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [98, 5003, 140001])
def test_large_upstream_gradients(vocab):
    """No factor on the way is larger than the gradient itself."""
    announce(f"large upstream gradients, vocabulary {vocab}")
    z, idx, val = far_rows(GAPS, vocab, 16, 1.0, F32, vocab)
    check(z, idx, val, 1.0, torch.full((len(GAPS),), 1e37))


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [98, 5003, 140001])
def test_loss_is_continuous_over_the_gap(vocab):
    gaps = [80.0 + 0.25 * i for i in range(48)]
    announce(f"loss over the gap, vocabulary {vocab}")
    z, idx, val = far_rows(gaps[:1], vocab, 16, 1.0, F32, 5)
    z, idx, val = [t.repeat(len(gaps), 1) for t in (z, idx, val)]
    z.scatter_add_(1, idx.long(), torch.tensor(gaps)[:, None].expand(-1, 16) - gaps[0])
    r = sgc.distill(z.cuda(), idx.cuda(), val.cuda(), mode=sgc.DISTILL_TAIL)
    u = 1.0 - float(val[0].double().exp().sum())
    rise = r.loss.cpu().double().diff()
    # 0.25 nats a step; a logit near 100 is rounded by 2^-18, the loss (below 100) by a few hundred U
    assert (rise - 0.25 * u).abs().max() < 2.0 ** -16 + 100 * 400 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,rows", [(98, 3), (5003, 3), (5003, 520), (140001, 3)], ids=str)
def test_nothing_left_outside(vocab, rows, dtype):
    """An outside that a mask has removed (-inf, the type's lowest value, 2^-1074 and less) has no
    tail, and one that holds a single live logit has all of it there."""
    announce(f"nothing left outside, {rows}x{vocab} {dtype}")
    z, idx, val = far_rows([10.0] * rows, vocab, 16, 1.0, dtype, 7)
    inside = torch.zeros(rows, vocab, dtype=torch.bool).scatter_(1, idx.long(), True)
    g = torch.ones(rows)
    for low in (-INF, torch.finfo(dtype).min, -2000.0):
        gone = torch.where(inside, z, torch.tensor(low, dtype=dtype))
        both = check(gone, idx, val, 1.0, g)
        assert (both.dlogits.cpu()[~inside] == 0).all()
        at = (~inside).int().argmax(1)
        one = gone.clone()
        one[torch.arange(rows), at] = -120.0
        if low != -2000.0:
            d = check(one, idx, val, 1.0, g).dlogits.cpu().double()
            u = 1.0 - val.double().exp().sum(1)
            off = (d[torch.arange(rows), at] + u).abs()
            # the rest is off by 70 U, then rounded
            assert (off < u * torch.finfo(dtype).eps + 80 * lm_tail_ref.U).all()


@pytest.mark.gpu
def test_broken_logits_inside_and_outside():
    """NaN and +inf, listed or not, make their own row NaN and no other."""
    for vocab in (98, 5003, 140001):
        announce(f"NaN and infinities, vocabulary {vocab}")
        z, idx, val = far_rows([100.0] * 5, vocab, 16, 1.0, F32, 3)
        inside = torch.zeros(5, vocab, dtype=torch.bool).scatter_(1, idx.long(), True)
        at = (~inside).int().argmax(1)
        for r, v in ((0, float("nan")), (1, INF)):
            z[r, at[r]] = v
        for r, v in ((2, float("nan")), (3, INF)):
            z[r, int(idx[r, 3])] = v
        r = sgc.distill(z.cuda(), idx.cuda(), val.cuda(), mode=sgc.DISTILL_TAIL, dloss=torch.ones(5, device="cuda"))
        assert torch.isnan(r.loss[:4]).all() and torch.isfinite(r.loss[4])
        assert torch.isnan(r.dlogits[:4]).any(1).all() and torch.isfinite(r.dlogits[4]).all()


@pytest.mark.gpu
def test_stats_of_ordinary_rows_are_plain_sums():
    """Without a far outside stats hold the sums at the row's maximum; such stats, made elsewhere, give the gradient."""
    announce("stats from elsewhere")
    for vocab in (98, 5003, 140001):
        z, idx, val = far_rows([0.0, 5.0, 12.0], vocab, 16, 1.0, F32, 9)
        x = z.double()
        m = x.amax(1, keepdim=True)
        e = (x - m).exp()
        want = torch.stack([m[:, 0], e.sum(1), e.scatter(1, idx.long(), 0.0).sum(1), torch.ones(3).double()], 1)
        i, v = idx.cuda(), val.cuda()
        got = sgc.distill(z.cuda(), i, v, mode=sgc.DISTILL_TAIL).stats.cpu().double()
        # the depth of the sums and 4 roundings of exponents of 30
        tol = want.abs() * lm_tail_ref.U * (lm_tail_ref.DEPTH + 4 * 30)
        assert ((got - want).abs() <= tol).all()
        z, idx, val = far_rows([25.0, 60.0, 80.0], vocab, 16, 1.0, F32, 9)
        x = z.double()
        m = x.amax(1, keepdim=True)
        e = (x - m).exp()
        st = torch.stack([m[:, 0], e.sum(1), e.scatter(1, idx.long(), 0.0).sum(1), torch.ones(3).double()], 1).float()
        g = torch.tensor([1.0, 65536.0, 1e30])
        _, d, _, td = lm_tail_ref.distill(z, idx, val, 1.0, g)
        close(sgc.distill_backward(z.cuda(), idx.cuda(), val.cuda(), st.cuda(), g.cuda(), mode=sgc.DISTILL_TAIL), d,
              td, "dlogits from stats made elsewhere", F32)
