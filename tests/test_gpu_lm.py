"""The language-model operators on the GPU against their 64-bit forms: types,
sizes from one element to long rows, strides and odd addresses, masks that
leave nothing, infinities and NaN in masked places, bad indices, streams,
graphs, in-place calls, and the same bits every time.
"""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm_ref
from gpu_util import announce
from lm_ref import close

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")
LOWEST = {t: torch.finfo(t).min for t in (F32, BF16, F16)}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_like(a, stride=None, offset=0):
    """a on the GPU with the given row stride, its first element `offset` past an aligned address."""
    rows, n = a.shape
    stride = n if stride is None else stride
    buf = torch.zeros(offset + max(rows - 1, 0) * stride + n + 8, dtype=a.dtype, device="cuda")
    v = buf.as_strided((rows, n), (stride, 1), offset)
    v.copy_(a)
    return v


def same_bits(a, b, what):
    for x, y in zip(a, b):
        if x is not None:
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)), what


# --------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (3, 2), (70, 100), (2049, 128), (33, 129), (5, 768), (5, 769), (5, 7), (2, 63), (1, 64), (9, 65), (33, 98), (4, 255), (130, 512), (7, 650),
               (300, 1000), (5, 1024), (3, 2047), (2, 2049), (600, 1031), (11, 4096), (6, 4099), (3, 8192), (2, 8200),
               (4, 16384), (2, 16385), (2, 40001), (1, 131075)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES, ids=str)
def test_norm(rows, cols, dtype):
    g = gen(rows * 7 + cols)
    x = (torch.randn(rows, cols, generator=g) * 1.5 + 0.5).to(dtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    w = torch.randn(cols, generator=g)
    b = torch.randn(cols, generator=g)
    announce(f"norm {rows}x{cols} {dtype}")
    eps = 1e-5
    xd, wd, bd = x.cuda(), w.cuda(), b.cuda()
    r = sgc.layer_norm(xd, wd, bd, eps=eps)
    (y, mean, rstd), (ty, tm, tr) = lm_ref.norm(x, w, b, eps)
    close(r.y, y, ty, "y", dtype)
    close(r.mean, mean, tm, "mean")
    close(r.rstd, rstd, tr, "rstd")
    gr = sgc.layer_norm_backward(dy.cuda(), xd, wd, r.mean, r.rstd)
    (dx, dw, db), (tdx, tdw, tdb) = lm_ref.norm_backward(dy, x, w, r.mean, r.rstd)
    close(gr.dx, dx, tdx, "dx", dtype)
    close(gr.dweight, dw, tdw, "dweight")
    close(gr.dbias, db, tdb, "dbias")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (4, 12)], ids=str)
@pytest.mark.parametrize("affine", ["both", "same", "none", "weight"])
def test_norm_strides_and_weights(dtype, offset, pad, affine):
    rows, cols = 37, 650
    g = gen(offset * 100 + pad)
    x = torch.randn(rows, cols, generator=g).to(dtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    wt = dtype if affine == "same" else F32
    w = None if affine == "none" else torch.randn(cols, generator=g).to(wt)
    b = None if affine in ("none", "weight") else torch.randn(cols, generator=g).to(wt)
    announce(f"norm strides {dtype} offset {offset} pad {pad} affine {affine}")
    xd = rows_like(x, cols + pad, offset)
    # the weight at an odd place, as a segment of a flat vector
    wd = None if w is None else rows_like(w[None], offset=1)[0]
    bd = None if b is None else rows_like(b[None], offset=3)[0]
    yd = rows_like(torch.zeros_like(x), cols + 2 * pad, 8 - offset)
    r = sgc.layer_norm(xd, wd, bd, out=yd)
    (y, mean, rstd), (ty, tm, tr) = lm_ref.norm(x, w, b, 1e-5)
    close(r.y, y, ty, "y", dtype)
    dyd = rows_like(dy, cols + pad + 1, offset + 1)
    dxd = rows_like(torch.zeros_like(x), cols + pad, offset)
    flat = torch.full((2 * cols + 5,), 7.0, device="cuda")
    gr = sgc.layer_norm_backward(dyd, xd, wd, r.mean, r.rstd, dx=dxd, dweight=flat[1:1 + cols],
                                 dbias=flat[cols + 2:2 * cols + 2])
    (dx, dw, db), (tdx, tdw, tdb) = lm_ref.norm_backward(dy, x, w, r.mean, r.rstd)
    close(gr.dx, dx, tdx, "dx", dtype)
    close(gr.dweight, dw, tdw, "dweight")
    close(gr.dbias, db, tdb, "dbias")
    assert [float(flat[k]) for k in (0, cols + 1, 2 * cols + 2, 2 * cols + 4)] == [7.0] * 4


def test_norm_adds_into_a_flat_gradient_and_in_place():
    rows, cols = 77, 1000
    g = gen(5)
    x, dy = torch.randn(rows, cols, generator=g), torch.randn(rows, cols, generator=g)
    w = torch.randn(cols, generator=g)
    announce("norm accumulate, in place")
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    r = sgc.layer_norm(xd, wd)
    one = sgc.layer_norm_backward(dyd, xd, wd, r.mean, r.rstd)
    flat = torch.randn(2 * cols, generator=g).cuda()
    was = flat.clone()
    sgc.layer_norm_backward(dyd, xd, wd, r.mean, r.rstd, dweight=flat[:cols], dbias=flat[cols:], accumulate=True,
                            want_dx=False)
    assert torch.equal(flat, was + torch.cat([one.dweight, one.dbias]))
    into_dy, into_x = dyd.clone(), xd.clone()
    sgc.layer_norm_backward(into_dy, xd, wd, r.mean, r.rstd, dx=into_dy)
    sgc.layer_norm_backward(dyd, into_x, wd, r.mean, r.rstd, dx=into_x)
    same_bits([into_dy, into_x], [one.dx, one.dx], "dx in place")
    y = xd.clone()
    sgc.layer_norm(y, wd, out=y)
    same_bits([y], [r.y], "y in place")
    for cols in (20000, 60001):  # rows longer than the registers hold
        x = torch.randn(3, cols, generator=g).cuda()
        r = sgc.layer_norm(x)
        y = x.clone()
        sgc.layer_norm(y, out=y)
        one = sgc.layer_norm_backward(x, x, None, r.mean, r.rstd)
        d = x.clone()
        sgc.layer_norm_backward(x, d, None, r.mean, r.rstd, dx=d)
        same_bits([y, d], [r.y, one.dx], f"in place, {cols} columns")


def test_norm_edges():
    announce("norm edges")
    e = torch.empty(0, 10, device="cuda")
    r = sgc.layer_norm(e)
    assert r.y.shape == (0, 10)
    flat = torch.full((20,), 3.0, device="cuda")
    sgc.layer_norm_backward(e, e, None, r.mean, r.rstd, dweight=flat[:10], dbias=flat[10:], accumulate=True)
    assert torch.equal(flat, torch.full_like(flat, 3.0))
    sgc.layer_norm_backward(e, e, None, r.mean, r.rstd, dweight=flat[:10], dbias=flat[10:])
    assert torch.equal(flat, torch.zeros_like(flat))
    # constant rows (variance 0), one input row for all (stride 0), a NaN row beside good ones
    x = torch.full((3, 100), 5.0)
    (y, mean, rstd), (ty, tm, tr) = lm_ref.norm(x, None, None, 1e-5)
    r = sgc.layer_norm(x.cuda())
    close(r.y, y, ty, "constant y")
    close(r.rstd, rstd, tr, "constant rstd")
    row = torch.randn(1, 300, generator=gen(1))
    r = sgc.layer_norm(row.cuda().expand(50, 300))
    (y, _, _), (ty, _, _) = lm_ref.norm(row.expand(50, 300), None, None, 1e-5)
    close(r.y, y, ty, "one row for all")
    x = torch.randn(4, 300, generator=gen(2))
    bad = x.clone()
    bad[2, 17] = NAN
    r, k = sgc.layer_norm(bad.cuda()), sgc.layer_norm(x.cuda())
    assert torch.isnan(r.y[2]).all()
    same_bits([r.y[:2], r.y[3]], [k.y[:2], k.y[3]], "rows beside a NaN row")


# ------------------------------------------------------- token log probabilities
def logits_for(rows, vocab, dtype, seed, kind):
    g = gen(seed)
    z = torch.randn(rows, vocab, generator=g) * 3
    if kind == "masked":
        z[torch.rand(rows, vocab, generator=g) < 0.4] = -INF
    z = z.to(dtype)
    if kind == "edges":
        for r in range(rows):
            k = r % 9
            if k == 0:
                z[r] = -INF                                   # nothing left
            elif k == 1:
                z[r] = LOWEST[dtype]                          # all masked by the lowest value
            elif k == 2:
                z[r, ::2] = LOWEST[dtype]
            elif k == 3:
                z[r] = 1.25                                   # all equal
            elif k == 4:
                z[r] = torch.linspace(-20, 20, vocab)         # ascending, with ties in 16 bits
            elif k == 5:
                z[r] = torch.linspace(20, -20, vocab)
            elif k == 6:
                z[r] = torch.where(torch.rand(vocab, generator=g) < 0.5, 0.0, -0.0)
            elif k == 7:
                z[r] = -INF
                z[r, vocab // 2] = -3.0                       # one token left
            else:
                z[r, vocab // 3] = 60000.0                    # one far above the rest
    if kind == "broken":
        for r in range(rows):
            if r % 3 == 0:
                z[r, vocab // 2] = NAN
            elif r % 3 == 1:
                z[r, vocab // 3] = INF
                z[r, vocab - 1] = INF
            else:
                z[r, 0] = -NAN
                z[r, vocab - 1] = INF
    return z


def check_logprobs(z, tokens, scale, top, zd=None, grads=True, **kw):
    rows, V = z.shape
    zd = z.cuda() if zd is None else zd
    td = None if tokens is None else tokens.cuda()
    r = sgc.token_logprobs(zd, td, scale=scale, top=top, **kw)
    sm, (logp, H, idx, tlp), (t_logp, t_H, t_tlp) = lm_ref.logprobs(z, tokens, scale, top)
    H = torch.where(sm.none, 0.0, H)
    close(r.entropy, H, t_H, "entropy")
    if tokens is not None:
        close(r.logp, logp, t_logp, "logp")
    if top:
        assert torch.equal(r.top_idx.cpu().long(), idx), "top_idx"
        close(r.top_logp, tlp, t_tlp, "top_logp")
    if not grads:
        return r
    g = torch.randn(rows, generator=gen(rows))
    h = torch.randn(rows, generator=gen(rows + 1))
    g[3::5], h[3::5] = 0.0, 0.0
    for gl, gh in ((g, h), (g, None), (None, h)):
        if gl is not None and tokens is None:
            continue
        d = sgc.token_logprobs_backward(zd, td, r.stats, r.entropy, None if gl is None else gl.cuda(),
                                        None if gh is None else gh.cuda(), scale=scale)
        ref, tol = lm_ref.logprobs_backward(sm, tokens, gl, gh)
        close(d, ref, tol, f"dlogits ({gl is not None}, {gh is not None})", z.dtype)
    return r


LP_SHAPES = [(1, 1, 1), (3, 2, 2), (4, 7, 5), (2, 63, 63), (9, 64, 20), (5, 65, 1), (70, 98, 16), (6, 255, 255),
             (5, 257, 256), (40, 1000, 5), (3, 2049, 64), (17, 4097, 20), (9, 10000, 256), (1, 10007, 20),
             (3, 50000, 20), (1, 131072, 64), (2, 131075, 8), (1, 300001, 100)]


def tokens_for(rows, vocab, seed, dtype=torch.int64):
    t = torch.randint(0, vocab, (rows,), generator=gen(seed)).to(dtype)
    t[2::4] = -1
    return t


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,top", LP_SHAPES, ids=str)
def test_logprobs(rows, vocab, top, dtype):
    announce(f"logprobs {rows}x{vocab} top {top} {dtype}")
    kind = "masked" if vocab > 300 and rows % 2 else "plain"
    z = logits_for(rows, vocab, dtype, rows + vocab, kind)
    check_logprobs(z, tokens_for(rows, vocab, vocab), 1.0 if vocab % 2 else 0.7, top)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,top", [(9, 9), (98, 20), (1003, 64), (5000, 256), (20011, 20)], ids=str)
@pytest.mark.parametrize("kind", ["edges", "broken"])
def test_logprobs_edges(kind, vocab, top, dtype):
    rows = 18 if kind == "edges" else 6
    announce(f"logprobs {kind} {rows}x{vocab} top {top} {dtype}")
    z = logits_for(rows, vocab, dtype, vocab, kind)
    check_logprobs(z, tokens_for(rows, vocab, 3, torch.int32), 1.5, top)


@pytest.mark.parametrize("vocab", [98, 40000, 300000])
def test_logprobs_edges_few_and_many_rows(vocab):
    """The same rows alone and among many: the ways of sharing the work give the same answers."""
    z = logits_for(18, vocab, BF16, 11, "edges")
    announce(f"logprobs few and many rows, vocabulary {vocab}")
    check_logprobs(z, None, 1.0, 40, grads=False)
    many = z.repeat(60, 1)
    r = check_logprobs(many[:18], None, 1.0, 40, grads=False)
    m = sgc.token_logprobs(many.cuda(), top=40)
    assert torch.equal(m.top_idx.view(60, 18, 40), r.top_idx.expand(60, 18, 40))
    same_bits([m.entropy[:18], m.top_logp[:18]], [m.entropy[18 * 59:], m.top_logp[18 * 59:]], "rows alike")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("offset,pad", [(0, 6), (1, 0), (3, 5), (4, 12)], ids=str)
@pytest.mark.parametrize("rows,vocab", [(5, 1001), (3, 30005)], ids=str)
def test_logprobs_strides(rows, vocab, offset, pad, dtype):
    announce(f"logprobs strides {rows}x{vocab} {dtype} offset {offset} pad {pad}")
    z = logits_for(rows, vocab, dtype, offset + pad, "masked")
    zd = rows_like(z, vocab + pad, offset)
    tok = tokens_for(rows, vocab, 4)
    r = check_logprobs(z, tok, 1.0, 10, zd=zd)
    g = torch.ones(rows, device="cuda")
    d = sgc.token_logprobs_backward(zd, tok.cuda(), r.stats, None, g)
    o = rows_like(torch.zeros_like(z), vocab + 2 * pad + 1, 7 - offset)
    sgc.token_logprobs_backward(zd, tok.cuda(), r.stats, None, g, dlogits=o)
    sgc.token_logprobs_backward(zd, tok.cuda(), r.stats, None, g, dlogits=zd)
    same_bits([o, zd], [d, d], "dlogits elsewhere, in place")


def test_logprobs_tokens_and_status():
    announce("logprobs bad tokens, no rows, one row for all")
    z = logits_for(6, 500, F32, 1, "plain")
    tok = torch.tensor([0, 499, 500, -1, -7, 1 << 40])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sgc.token_logprobs(z.cuda(), tok.cuda(), status=st)
    assert int(st) == sgc.STATUS_BAD_INPUT
    lp = r.logp.cpu()
    assert torch.isnan(lp[[2, 5]]).all() and (lp[[3, 4]] == 0).all() and torch.isfinite(lp[:2]).all()
    d = sgc.token_logprobs_backward(z.cuda(), tok.cuda(), r.stats, None, torch.ones(6, device="cuda"))
    assert (d[2:] == 0).all() and (d[:2] != 0).any()
    st.zero_()
    sgc.token_logprobs(z.cuda(), tok[:2].repeat(3).cuda(), status=st)
    assert int(st) == 0
    e = sgc.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top=3)
    assert e.logp.shape == (0,) and e.top_idx.shape == (0, 3)
    one = z[:1].cuda().expand(40, 500)
    m = check_logprobs(z[:1].expand(40, 500), tok[:1].repeat(40), 1.0, 4, zd=one)
    same_bits([m.logp[:1]], [m.logp[39:]], "one row for all")


def test_rows_past_32_bits():
    """The second row starts past 2^31 elements and 2^32 bytes."""
    V, k = 5003, 6
    stride = (1 << 31) + 16
    announce("offsets past 32 bits")
    buf = torch.zeros(stride + V, dtype=BF16, device="cuda")
    z = logits_for(2, V, BF16, 5, "plain")
    zd = buf.as_strided((2, V), (stride, 1))
    zd.copy_(z)
    check_logprobs(z, torch.tensor([7, 5002]), 1.0, 20, zd=zd)
    idx = torch.stack([torch.randperm(V, generator=gen(r))[:k] for r in range(2)]).int()
    val = torch.log_softmax(torch.randn(2, 2 * k, generator=gen(8)), 1)[:, :k].contiguous()
    loss, d, tl, td = lm_ref.distill(z, idx, val, True, 1.0)
    r = sgc.distill(zd, idx.cuda(), val.cuda(), mode=sgc.DISTILL_TAIL, dlogits=zd)
    close(r.loss, loss, tl, "loss")
    close(zd, d, td, "dlogits", BF16)
    zd.copy_(z)
    n = sgc.layer_norm(zd)
    (y, _, _), (ty, _, _) = lm_ref.norm(z, None, None, 1e-5)
    close(n.y, y, ty, "y", BF16)
    gr = sgc.layer_norm_backward(n.y, zd, None, n.mean, n.rstd, dx=zd)
    (dx, dw, _), (tdx, tdw, _) = lm_ref.norm_backward(n.y, z, None, n.mean, n.rstd)
    close(zd, dx, tdx, "dx", BF16)
    close(gr.dweight, dw, tdw, "dweight")


# ------------------------------------------------------------ distillation
def entries_for(z, k, seed, tail, kind="plain"):
    rows, V = z.shape
    g = gen(seed)
    n = min(k, V)
    idx = torch.full((rows, k), -1, dtype=torch.int32)
    for r in range(rows):
        at = torch.randperm(V, generator=g)[:n] if V < 4096 else \
            torch.randint(0, V // n, (n,), generator=g) + torch.arange(n) * (V // n)
        idx[r, torch.randperm(k, generator=g)[:n]] = at[torch.randperm(n, generator=g)].int()
    v = torch.randn(rows, k, generator=g) * 2
    if tail:
        mass = torch.rand(rows, 1, generator=g) * 0.4 + 0.5
        v = torch.log_softmax(torch.where(idx < 0, -INF, v), 1) + mass.log()
    v = torch.where(idx < 0, 123.0, v)                  # what an absent entry holds does not count
    if kind == "ragged":
        for r in range(rows):
            if r % 4 == 0:
                idx[r] = -1                             # no entry at all
            elif r % 4 == 1:
                idx[r, 1:] = -1
            elif r % 4 == 2:
                v[r, ::2] = -INF                        # entries of no probability
    return idx, v


def check_distill(z, idx, val, tail, scale=1.0, teacher_scale=1.0, zd=None):
    rows, V = z.shape
    mode = sgc.DISTILL_TAIL if tail else sgc.DISTILL_RENORM
    kw = dict(mode=mode, scale=scale, teacher_scale=teacher_scale)
    zd = z.cuda() if zd is None else zd
    g = torch.rand(rows, generator=gen(V)) + 0.5
    g[5::7] = 0.0
    loss, d, tl, td = lm_ref.distill(z, idx, val, tail, scale, teacher_scale, g)
    i, v, gd = idx.cuda(), val.cuda(), g.cuda()
    one = sgc.distill(zd, i, v, **kw)
    close(one.loss, loss, tl, "loss")
    assert one.dlogits is None
    both = sgc.distill(zd, i, v, dloss=gd, **kw)
    close(both.loss, loss, tl, "loss of the call with the gradient")
    close(both.dlogits, d, td, "dlogits of the loss call", z.dtype)
    back = sgc.distill_backward(zd, i, v, one.stats, gd, **kw)
    close(back, d, td, "dlogits of the backward call", z.dtype)
    return one, both, back


DI_SHAPES = [(1, 1, 1), (3, 2, 4), (4, 7, 5), (2, 63, 63), (9, 64, 80), (70, 98, 16), (5, 257, 256), (40, 1000, 8),
             (3, 2049, 64), (17, 4097, 32), (600, 1001, 20), (9, 10000, 256), (1, 10007, 50), (3, 50000, 64),
             (300, 20001, 40), (1, 131072, 128), (2, 131075, 8), (1, 300001, 100)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("rows,vocab,k", DI_SHAPES, ids=str)
def test_distill(rows, vocab, k, tail, dtype):
    announce(f"distill {rows}x{vocab} top {k} {dtype} tail {tail}")
    z = logits_for(rows, vocab, dtype, rows + vocab, "plain")
    idx, val = entries_for(z, k, vocab + k, tail)
    check_distill(z, idx, val, tail, scale=1.0 if vocab % 2 else 0.5, teacher_scale=1.0 if tail else 0.5)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
@pytest.mark.parametrize("kind", ["ragged", "edges", "masked", "broken"])
@pytest.mark.parametrize("vocab,k", [(98, 16), (1003, 64), (20011, 20)], ids=str)
def test_distill_edges(vocab, k, kind, tail, dtype):
    rows = 18
    announce(f"distill {kind} {rows}x{vocab} top {k} {dtype} tail {tail}")
    z = logits_for(rows, vocab, dtype, vocab, "plain" if kind == "ragged" else kind)
    idx, val = entries_for(z, k, k, tail, kind)
    if kind in ("edges", "masked"):
        # a teacher gives nothing to what its student may not say
        at = idx.long().clamp(min=0)
        hidden = z.float().gather(1, at) <= LOWEST[dtype] / 2
        val = torch.where(hidden & (idx >= 0), -INF, val)
    check_distill(z, idx, val, tail, scale=0.75)


@pytest.mark.parametrize("vocab", [98, 3001, 40004, 150001])
def test_logits_far_from_zero(vocab):
    """Maxima of 1e4 to 3e38 either way, alone in their row or with an ordinary rest."""
    rows = 600 if vocab < 5000 else 12
    announce(f"logits far from zero, {rows}x{vocab}")
    z = torch.randn(rows, vocab, generator=gen(vocab))
    for r in range(rows):
        far = (1e4, -1e4, 7e7, -7e7, 3e8, -3e8, 1e12, -1e12, 1e30, -1e30, 3e38, -3e38)[r % 12]
        if r % 24 < 12:
            z[r] = far + z[r] * max(1.0, abs(far) * 1e-7)
        else:
            z[r, vocab // 2] = far
    check_logprobs(z, tokens_for(rows, vocab, 3), 1.0, 10)
    idx, val = entries_for(z, 12, 3, True)
    for tail in (False, True):
        # entries far below their row's maximum would have an infinite loss
        near = z.gather(1, idx.long().clamp(min=0)) > z.amax(1, keepdim=True) - 80
        check_distill(z, idx, torch.where(near, val, -INF), tail)


def test_distill_student_without_the_teachers_token():
    announce("distill: the student gives a taught token nothing")
    z = torch.randn(2, 500, generator=gen(1))
    z[0, 40] = -INF
    idx = torch.tensor([[40, 3], [40, 3]], dtype=torch.int32)
    val = torch.tensor([[-0.5, -1.0], [-0.5, -1.0]])
    for tail in (False, True):
        check_distill(z, idx, val, tail)
    r = sgc.distill(z.cuda(), idx.cuda(), val.cuda())
    assert float(r.loss[0]) == INF


def test_distill_bad_rows():
    announce("distill: bad rows")
    rows, V, k = 6, 700, 5
    z = torch.randn(rows, V, generator=gen(1))
    idx, val = entries_for(z, k, 3, True)
    idx[1, 2] = V
    idx[2, 0] = -2
    idx[3, 4] = idx[3, 1]
    idx[4, 0] = 2 ** 31 - 1
    for tail in (False, True):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        mode = sgc.DISTILL_TAIL if tail else sgc.DISTILL_RENORM
        r = sgc.distill(z.cuda(), idx.cuda(), val.cuda(), mode=mode, dloss=torch.ones(rows, device="cuda"), status=st)
        assert int(st) == sgc.STATUS_CORRUPT
        assert torch.isnan(r.loss[1:5]).all() and torch.isfinite(r.loss[[0, 5]]).all()
        assert (r.dlogits[1:5] == 0).all() and (r.dlogits[[0, 5]] != 0).any(1).all()
        d = sgc.distill_backward(z.cuda(), idx.cuda(), val.cuda(), r.stats, mode=mode)
        assert torch.equal(d, r.dlogits)
        check_distill(z, idx, val, tail)
    # the same on rows that are split over workgroups
    z = torch.randn(3, 200003, generator=gen(2))
    idx = torch.tensor([[5, 150000, 5], [5, 150000, 200003], [200002, 0, 77]], dtype=torch.int32)
    val = torch.full((3, 3), -2.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sgc.distill(z.cuda(), idx.cuda(), val.cuda(), mode=sgc.DISTILL_TAIL, status=st)
    assert int(st) == sgc.STATUS_CORRUPT
    assert torch.isnan(r.loss[:2]).all() and torch.isfinite(r.loss[2])
    check_distill(z, idx, val, True)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab", [(5, 1001), (3, 30005), (700, 2003)], ids=str)
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 5), (4, 12)], ids=str)
def test_distill_strides_and_in_place(rows, vocab, offset, pad, dtype):
    announce(f"distill strides {rows}x{vocab} {dtype} offset {offset} pad {pad}")
    z = logits_for(rows, vocab, dtype, offset, "plain")
    idx, val = entries_for(z, 20, 9, True)
    zd = rows_like(z, vocab + pad, offset)
    one, both, back = check_distill(z, idx, val, True, zd=zd)
    g = (torch.rand(rows, generator=gen(vocab)) + 0.5)
    g[5::7] = 0.0
    kw = dict(mode=sgc.DISTILL_TAIL)
    o = rows_like(torch.zeros_like(z), vocab + 2 * pad + 1, 7 - offset)
    sgc.distill(zd, idx.cuda(), val.cuda(), dloss=g.cuda(), dlogits=o, **kw)
    a, b = rows_like(z, vocab + pad, offset), rows_like(z, vocab + pad, offset)
    sgc.distill(a, idx.cuda(), val.cuda(), dloss=g.cuda(), dlogits=a, **kw)
    sgc.distill_backward(b, idx.cuda(), val.cuda(), one.stats, g.cuda(), dlogits=b, **kw)
    same_bits([o, a, b], [both.dlogits, both.dlogits, back], "dlogits elsewhere, in place")


def test_distill_gradient_against_differences():
    """The kernel's fp32 gradient against central differences of the 64-bit loss."""
    announce("distill, logprobs: gradients against differences")
    z = torch.randn(2, 40, generator=gen(6))
    idx, val = entries_for(z, 6, 2, True)
    tok = torch.tensor([3, 39])
    for tail in (False, True):
        mode = sgc.DISTILL_TAIL if tail else sgc.DISTILL_RENORM
        d = sgc.distill(z.cuda(), idx.cuda(), val.cuda(), mode=mode, scale=0.8,
                        dloss=torch.ones(2, device="cuda")).dlogits.cpu().double()
        check_differences(d, z, lambda x: lm_ref.distill(x, idx, val, tail, 0.8)[0].sum())
    r = sgc.token_logprobs(z.cuda(), tok.cuda(), scale=0.8)
    d = sgc.token_logprobs_backward(z.cuda(), tok.cuda(), r.stats, r.entropy, torch.ones(2, device="cuda"),
                                    torch.ones(2, device="cuda"), scale=0.8).cpu().double()
    check_differences(d, z, lambda x: sum(lm_ref.logprobs(x, tok, 0.8, 0)[1][k].sum() for k in (0, 1)))


def check_differences(d, z, f):
    z = z.double()
    for i in range(z.numel()):
        hi, lo = z.clone(), z.clone()
        hi.view(-1)[i] += 1e-4
        lo.view(-1)[i] -= 1e-4
        want = float((f(hi) - f(lo)) / 2e-4)
        # differences: (1e-4)^2 times a third derivative below 2; the kernel: a few hundred U of terms below 2
        assert abs(float(d.view(-1)[i]) - want) < 2e-8 + 400 * lm_ref.U, i


# ---------------------------------------------------------- how it is called
def step_tensors(rows=64, vocab=20000, cols=512):
    g = gen(42)
    z = (torch.randn(rows, vocab, generator=g) * 2).to(BF16)
    x = torch.randn(rows, cols, generator=g)
    idx, val = entries_for(z, 32, 1, True)
    return [t.cuda() for t in (z, x, tokens_for(rows, vocab, 1), idx, val, torch.rand(rows, generator=g))]


def all_calls(z, x, tok, idx, val, g, ws=None, stream=None, scale_in=1.0):
    ws = ws or [None] * 3
    n = sgc.layer_norm(x, stream=stream)
    nb = sgc.layer_norm_backward(x, x, None, n.mean, n.rstd, ws=ws[0], stream=stream)
    lp = sgc.token_logprobs(z, tok, top=20, ws=ws[1], stream=stream)
    lb = sgc.token_logprobs_backward(z, tok, lp.stats, lp.entropy, g, g, stream=stream)
    di = sgc.distill(z, idx, val, mode=sgc.DISTILL_TAIL, dloss=g, ws=ws[2], stream=stream)
    db = sgc.distill_backward(z, idx, val, di.stats, g, mode=sgc.DISTILL_TAIL, stream=stream)
    return [n.y, n.mean, n.rstd, nb.dx, nb.dweight, nb.dbias, lp.logp, lp.entropy, lp.stats, lp.top_idx, lp.top_logp,
            lb, di.loss, di.stats, di.dlogits, db]


def workspaces(rows, vocab, cols, fill):
    sizes = [sgc.layer_norm_backward_workspace_bytes(rows, cols),
             sgc.token_logprobs_workspace_bytes(rows, vocab, top=20, dtype=BF16),
             sgc.distill_workspace_bytes(rows, vocab, 32, dtype=BF16)]
    return [torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda") for n in sizes]


@pytest.mark.parametrize("rows,vocab,cols", [(64, 20000, 512), (2, 150000, 650), (700, 98, 4096)], ids=str)
def test_same_bits_whatever_the_workspace_held(rows, vocab, cols):
    announce(f"same bits {rows}x{vocab}")
    a = step_tensors(rows, vocab, cols)
    first = all_calls(*a)
    for fill in (0, 0x5A, 0xFF):
        same_bits(all_calls(*a, ws=workspaces(rows, vocab, cols, fill)), first, f"workspace of {fill}")


def test_streams():
    announce("streams")
    a = step_tensors()
    first = all_calls(*a)
    s = torch.cuda.Stream()
    z = torch.empty_like(a[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        z.copy_(a[0])  # the call has to wait for this: same stream
        other = all_calls(z, *a[1:], stream=s)
    s.synchronize()
    same_bits(other, first, "another stream")


@pytest.mark.parametrize("rows,vocab,cols", [(64, 20000, 512), (2, 150000, 650)], ids=str)
def test_graph_replays(rows, vocab, cols):
    announce(f"graph {rows}x{vocab}")
    a = step_tensors(rows, vocab, cols)
    ws = workspaces(rows, vocab, cols, 0)
    z_in, x_in = a[0].clone(), a[1].clone()
    all_calls(z_in, x_in, *a[2:], ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(z_in, x_in, *a[2:], ws=ws)
    torch.cuda.synchronize()
    for it in range(4):
        z_in.copy_(torch.roll(a[0], it, 1))
        x_in.copy_(a[1] * (1 + it))
        want = all_calls(z_in, x_in, *a[2:])  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same_bits(out, want, f"replay {it}")


def test_captured_call_needs_its_own_workspace():
    announce("a captured call without a workspace is refused")
    z = torch.randn(1, 400000, device="cuda")
    if sgc.token_logprobs_workspace_bytes(1, 400000, top=4) == sgc.lm.LM_WS_NONE:
        pytest.skip("no workspace at this size")
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError):
        with torch.cuda.graph(graph):
            sgc.token_logprobs(z, top=4)
    torch.cuda.synchronize()


def test_top_list_of_a_teacher_is_what_distill_takes():
    """token_logprobs' top list goes straight into distill: a student equal to its teacher has no loss."""
    announce("teacher's list")
    z = (torch.randn(50, 10000, generator=gen(3)) * 2).cuda()
    t = sgc.token_logprobs(z, top=64)
    r = sgc.distill(z, t.top_idx, t.top_logp, mode=sgc.DISTILL_TAIL, dloss=torch.ones(50, device="cuda"))
    # both sides' terms are below 16; their errors a few hundred U
    assert float(r.loss.abs().max()) < 16 * 400 * lm_ref.U
    assert float(r.dlogits.abs().max()) < 400 * lm_ref.U


# ------------------------------------------------- large calls, many rows
def big_rows(vocab, dtype, both=2):
    """So many rows that a call moves more than the last-level cache holds."""
    return (256 << 20) // (both * vocab * dtype.itemsize) + 3


@pytest.mark.parametrize("vocab,dtype", [(5003, BF16), (20016, BF16), (50001, F16), (50008, BF16), (40004, F32),
                                         (65536, BF16), (130072, BF16), (131072, BF16), (70001, F32)], ids=str)
@pytest.mark.parametrize("tail", [False, True], ids=["renorm", "tail"])
def test_large_distill(vocab, dtype, tail):
    rows = big_rows(vocab, dtype)
    announce(f"large distill {rows}x{vocab} {dtype} tail {tail}")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.empty(rows, vocab, dtype=dtype, device="cuda").normal_(0.0, 3.0, generator=g)
    k, pick = 24, torch.tensor([0, 1, 2, 3, rows // 2, rows - 2, rows - 1])
    idx, val = entries_for(z[:64].cpu(), k, 5, tail)
    idx, val = [t.repeat(-(-rows // 64), 1)[:rows].contiguous() for t in (idx, val)]
    dl = torch.rand(rows, generator=gen(2)) + 0.5
    dl[2] = 0.0
    mode = sgc.DISTILL_TAIL if tail else sgc.DISTILL_RENORM
    r = sgc.distill(z, idx.cuda(), val.cuda(), mode=mode, dloss=dl.cuda())
    b = sgc.distill_backward(z, idx.cuda(), val.cuda(), r.stats, dl.cuda(), mode=mode)
    loss, d, tl, td = lm_ref.distill(z[pick].cpu(), idx[pick], val[pick], tail, 1.0, g=dl[pick])
    close(r.loss[pick], loss, tl, "loss")
    close(r.dlogits[pick], d, td, "dlogits", dtype)
    close(b[pick], d, td, "dlogits of the backward call", dtype)
    in_place = sgc.distill(z, idx.cuda(), val.cuda(), mode=mode, dloss=dl.cuda(), dlogits=z)
    same_bits([in_place.dlogits, in_place.loss], [r.dlogits, r.loss], "in place")


@pytest.mark.parametrize("vocab,dtype", [(1000, BF16), (20016, BF16), (50001, F16), (40004, F32), (131072, BF16)],
                         ids=str)
def test_large_logprobs(vocab, dtype):
    rows = big_rows(vocab, dtype, 1)
    announce(f"large logprobs {rows}x{vocab} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.empty(rows, vocab, dtype=dtype, device="cuda").normal_(0.0, 3.0, generator=g)
    z[1, ::2] = -INF
    pick = torch.tensor([0, 1, 2, 3, rows // 2, rows - 2, rows - 1])
    tok = tokens_for(rows, vocab, 3)
    r = sgc.token_logprobs(z, tok.cuda(), top=20)
    sm, (logp, H, at, tlp), (t_logp, t_H, t_tlp) = lm_ref.logprobs(z[pick].cpu(), tok[pick], 1.0, 20)
    close(r.logp[pick], logp, t_logp, "logp")
    close(r.entropy[pick], H, t_H, "entropy")
    assert torch.equal(r.top_idx[pick].cpu().long(), at)
    close(r.top_logp[pick], tlp, t_tlp, "top_logp")
    gl, gh = torch.randn(rows, generator=gen(1)), torch.randn(rows, generator=gen(2))
    gl[3] = gh[3] = 0.0
    for h in (gh, None):
        d = sgc.token_logprobs_backward(z, tok.cuda(), r.stats, r.entropy, gl.cuda(), None if h is None else h.cuda())
        ref, tol = lm_ref.logprobs_backward(sm, tok[pick], gl[pick], None if h is None else h[pick])
        close(d[pick], ref, tol, "dlogits", dtype)


@pytest.mark.parametrize("cols,dtype", [(98, BF16), (650, F32), (1000, F16), (2048, BF16), (4099, BF16), (8192, F16),
                                        (12000, BF16), (16384, F32), (20000, BF16)], ids=str)
def test_large_norm(cols, dtype):
    rows = big_rows(cols, dtype)
    announce(f"large norm {rows}x{cols} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(0.5, 1.5, generator=g)
    dy = torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=g)
    w, b = torch.randn(cols, generator=gen(1)), torch.randn(cols, generator=gen(2))
    pick = torch.tensor([0, 1, 2, 3, rows // 2, rows - 2, rows - 1])
    r = sgc.layer_norm(x, w.cuda(), b.cuda())
    (y, mean, rstd), (ty, tm, tr) = lm_ref.norm(x[pick].cpu(), w, b, 1e-5)
    close(r.y[pick], y, ty, "y", dtype)
    close(r.mean[pick], mean, tm, "mean")
    close(r.rstd[pick], rstd, tr, "rstd")
    gr = sgc.layer_norm_backward(dy, x, w.cuda(), r.mean, r.rstd)
    (dx, _, _), (tdx, _, _) = lm_ref.norm_backward(dy[pick].cpu(), x[pick].cpu(), w, r.mean[pick], r.rstd[pick])
    close(gr.dx[pick], dx, tdx, "dx", dtype)
    # the sums over the rows, in 64 bits on the GPU: rows one after the other in a part, then the parts
    dw, db, aw, ab, tw = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(5))
    for a in range(0, rows, 8192):
        s = slice(a, a + 8192)
        d64 = dy[s].double()
        h = (x[s].double() - r.mean[s].double()[:, None]) * r.rstd[s].double()[:, None]
        dw, db = dw + (d64 * h).sum(0), db + d64.sum(0)
        aw, ab = aw + (d64 * h).abs().sum(0), ab + d64.abs().sum(0)
        tw = tw + (d64.abs() * (2 * (x[s].double().abs() + r.mean[s].double().abs()[:, None])
                                * r.rstd[s].double()[:, None] + h.abs())).sum(0)
    deep = lm_ref.DEPTH + min(rows, 512) + rows // 64
    close(gr.dweight, dw.cpu(), (lm_ref.U * ((deep + 2) * aw + tw)).cpu(), "dweight")
    close(gr.dbias, db.cpu(), (lm_ref.U * deep * ab).cpu(), "dbias")
    only = sgc.layer_norm_backward(dy, x, w.cuda(), r.mean, r.rstd, want_dx=False)
    same_bits([only.dweight, only.dbias], [gr.dweight, gr.dbias], "sums alone")


def test_more_rows_than_a_grid_line():
    """Rows past 2^20, where the grid gets a second line; every row is checked."""
    rows, V = (1 << 20) + 3, 5
    announce(f"{rows} rows of {V}")
    z = torch.randn(rows, V, generator=gen(1)) * 3
    check_logprobs(z, tokens_for(rows, V, 2), 1.0, 2)
    idx = torch.stack([torch.randint(0, 2, (rows,), generator=gen(3)),
                       torch.randint(2, V, (rows,), generator=gen(4))], 1).int()
    val = torch.log_softmax(torch.randn(rows, 3, generator=gen(5)), 1)[:, :2].contiguous()
    check_distill(z, idx, val, True)
    r = sgc.layer_norm(z.cuda())
    (y, _, _), (ty, _, _) = lm_ref.norm(z, None, None, 1e-5)
    close(r.y, y, ty, "y")


@pytest.mark.parametrize("vocab", [98, 5003, 150001])
def test_distill_ignores_what_absent_entries_hold(vocab):
    rows = 600 if vocab < 6000 else 4
    announce(f"distill: NaN and infinities in absent entries, {rows}x{vocab}")
    z = torch.randn(rows, vocab, generator=gen(vocab)).cuda()
    for tail in (False, True):
        idx, val = entries_for(z.cpu(), 12, 7, tail)
        idx[:, 5] = -1
        mode = sgc.DISTILL_TAIL if tail else sgc.DISTILL_RENORM
        out = []
        for junk in (0.0, NAN, INF, -INF):
            val[:, 5] = junk
            r = sgc.distill(z, idx.cuda(), val.cuda(), mode=mode, dloss=torch.ones(rows, device="cuda"))
            assert torch.isfinite(r.loss).all()
            out.append([r.loss, r.dlogits])
        for o in out[1:]:
            same_bits(o, out[0], "what an absent entry holds")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab,k", [(2049, 32), (5003, 5), (12288, 33)], ids=str)
@pytest.mark.parametrize("kind", ["edges", "masked", "broken"])
def test_many_short_rows(kind, vocab, k, dtype):
    rows = 520
    announce(f"{kind} {rows}x{vocab} top {k} {dtype}")
    z = logits_for(rows, vocab, dtype, vocab, kind)
    check_logprobs(z, tokens_for(rows, vocab, 3, torch.int32), 1.5, k)
    for tail in (False, True):
        idx, val = entries_for(z, k, k, tail, kind)
        if kind != "broken":
            # a teacher gives nothing to what its student may not say
            hidden = z.float().gather(1, idx.long().clamp(min=0)) <= LOWEST[dtype] / 2
            val = torch.where(hidden & (idx >= 0), -INF, val)
        check_distill(z, idx, val, tail, scale=0.75)
