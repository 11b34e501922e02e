"""RMS norm, rows in 8 bits and products of 8-bit integers on the GPU against
their plain forms: types, sizes from one element to long rows, strides and odd
addresses, values that are not finite, in-place calls, buffers' surroundings,
streams, graphs, and the same bits every time.
"""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm8_ref
import lm_ref
from gpu_util import announce
from lm_ref import close, dbl

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["fp32", "bf16", "fp16"])
INF, NAN = float("inf"), float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows_like(a, stride=None, offset=0, fill=7):
    """a on the GPU at the given row stride, its first element `offset` past an aligned address, and the buffer."""
    rows, n = a.shape
    stride = n if stride is None else stride
    buf = torch.full((offset + max(rows - 1, 0) * stride + n + 40,), fill, dtype=a.dtype, device="cuda")
    v = buf.as_strided((rows, n), (stride, 1), offset)
    v.copy_(a)
    return v, buf


def untouched(v, buf, fill=7):
    """Everything of the buffer outside v still holds what it did."""
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(True)
    assert bool((buf[~inside] == fill).all()), "written outside its rows"


def same_bits(a, b, what):
    for x, y in zip(a, b):
        if x is not None:
            x, y = x.contiguous(), y.contiguous()
            assert x.dtype == y.dtype and torch.equal(x.view(torch.uint8), y.view(torch.uint8)), what


def equal_bits(got, want, what):
    """The same bits, any NaN for a NaN."""
    got = got.detach().cpu()
    assert got.dtype == want.dtype and got.shape == want.shape, what
    if got.is_floating_point():
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan), f"{what}: NaN at other places"
        got, want = torch.where(nan, 0.0, got), torch.where(nan, 0.0, want)
    assert torch.equal(got, want), f"{what}: {int((got != want).sum())} of {got.numel()} differ"


# ----------------------------------------------------------------- RMS norm
SHAPES = [(1, 1), (3, 2), (70, 100), (2049, 128), (33, 129), (5, 513), (5, 768), (5, 769), (5, 7), (2, 63), (1, 64),
          (9, 65), (33, 98), (4, 255), (130, 512), (7, 650), (300, 1000), (5, 1024), (3, 2047), (2, 2049), (600, 1031),
          (4, 1300), (11, 4096), (6, 4099), (3, 8192), (2, 8200), (4, 16384), (2, 16385), (2, 40001), (1, 131075)]


def stream_rows(rows, cols, dtype, g):
    loud = torch.where(torch.rand(cols, generator=g) < 0.02, 8.0, 1.0)
    return (torch.randn(rows, cols, generator=g) * loud).to(dtype)


@DTYPES
@pytest.mark.parametrize("rows,cols", SHAPES, ids=str)
def test_rms(rows, cols, dtype):
    g = gen(rows * 7 + cols)
    x, res, w = stream_rows(rows, cols, dtype, g), torch.randn(rows, cols, generator=g).to(dtype), \
        torch.randn(cols, generator=g)
    dy, ds = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    announce(f"rms {rows}x{cols} {dtype}")
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()
    for residual in (None, res):
        s = lm8_ref.stream(x, residual)
        r = sgc.rms_norm(xd, wd, residual=None if residual is None else rd)
        equal_bits(r.sum, s, "sum")
        (y, rstd), (ty, tr) = lm8_ref.rms(s, w, 1e-6)
        close(r.y, y, ty, "y", dtype)
        close(r.rstd, rstd, tr, "rstd")
        q = sgc.rms_norm_q8(xd, wd, residual=None if residual is None else rd)
        equal_bits(q.sum, s, "sum beside 8 bits")
        want, (scale, rstd), (ts, tr) = lm8_ref.rms_q8(s, w, 1e-6)
        equal_bits(q.q8.q, want, "q")
        close(q.q8.scale, scale, ts, "scale")
        close(q.rstd, rstd, tr, "rstd beside 8 bits")
        b = sgc.rms_norm_backward(dy.cuda(), r.sum, wd, r.rstd, dsum=None if residual is None else ds.cuda())
        (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, s, w, None, r.rstd, None if residual is None else ds)
        close(b.dx, dx, tdx, "dx", dtype)
        close(b.dweight, dw, tdw, "dweight")


@DTYPES
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (4, 12)], ids=str)
@pytest.mark.parametrize("cols", [100, 650, 1031, 4096])
@pytest.mark.parametrize("weight", ["fp32", "same", "none"])
def test_rms_strides_and_weights(dtype, offset, pad, cols, weight):
    rows = 37
    g = gen(offset * 100 + pad + cols)
    x, res, dy, ds = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(4)]
    w = None if weight == "none" else torch.randn(cols, generator=g).to(dtype if weight == "same" else F32)
    announce(f"rms strides {dtype} cols {cols} offset {offset} pad {pad} weight {weight}")
    xd, rd = rows_like(x, cols + pad, offset)[0], rows_like(res, cols + 3, offset + 1)[0]
    wd = None if w is None else rows_like(w[None], offset=1)[0][0]
    s = lm8_ref.stream(x, res)
    (sd, sbuf), (yd, ybuf) = rows_like(s * 0, cols + pad + 1, 5), rows_like(s * 0, cols + 2 * pad, 8 - offset)
    r = sgc.rms_norm(xd, wd, residual=rd, out=yd, sum_out=sd, eps=1e-3)
    (y, rstd), (ty, tr) = lm8_ref.rms(s, w, 1e-3)
    equal_bits(r.sum, s, "sum")
    close(r.y, y, ty, "y", dtype)
    untouched(sd, sbuf)
    untouched(yd, ybuf)
    qd, qbuf = rows_like(torch.zeros(rows, cols, dtype=torch.int8), cols + pad, offset)
    out = sgc.Quantized(qd, torch.empty(rows, 1, device="cuda"))
    q = sgc.rms_norm_q8(xd, wd, residual=rd, eps=1e-3, out=out)
    want, (scale, _), (ts, _) = lm8_ref.rms_q8(s, w, 1e-3)
    equal_bits(q.q8.q, want, "q")
    close(q.q8.scale, scale, ts, "scale")
    untouched(qd, qbuf)
    dyd, dsd = rows_like(dy, cols + pad + 1, offset + 1)[0], rows_like(ds, cols + 2, 3)[0]
    dxd, dxbuf = rows_like(s * 0, cols + pad, offset)
    flat = torch.full((cols + 4,), 7.0, device="cuda")
    b = sgc.rms_norm_backward(dyd, sd, wd, r.rstd, dsum=dsd, dx=dxd, dweight=flat[1:1 + cols])
    (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, s, w, None, r.rstd, ds)
    close(b.dx, dx, tdx, "dx", dtype)
    close(b.dweight, dw, tdw, "dweight")
    untouched(dxd, dxbuf)
    assert flat[0] == 7.0 and flat[cols + 1] == 7.0


@pytest.mark.parametrize("cols", [96, 1000, 4096, 20000])
def test_rms_in_place_and_added(cols):
    rows = 77
    g = gen(cols)
    x, res, dy, ds = [torch.randn(rows, cols, generator=g).to(BF16).cuda() for _ in range(4)]
    w = torch.randn(cols, generator=g).cuda()
    announce(f"rms in place, {cols} columns")
    r = sgc.rms_norm(x, w, residual=res)
    q = sgc.rms_norm_q8(x, w, residual=res)
    for sum_at, y_at in (("x", "res"), ("res", "x"), ("x", None), (None, "x"), ("res", None), (None, "res")):
        t = dict(x=x.clone(), res=res.clone())
        got = sgc.rms_norm(t["x"], w, residual=t["res"], sum_out=t.get(sum_at), out=t.get(y_at))
        same_bits([got.y, got.sum, got.rstd], [r.y, r.sum, r.rstd], f"sum in {sum_at}, y in {y_at}")
        got = sgc.rms_norm_q8(t["x"] if y_at is None and sum_at is None else x.clone(), w, residual=res)
        same_bits([got.q8.q, got.q8.scale], [q.q8.q, q.q8.scale], "8 bits")
    t = x.clone()
    got = sgc.rms_norm_q8(t, w, residual=res, sum_out=t)
    same_bits([got.q8.q, got.q8.scale, t], [q.q8.q, q.q8.scale, q.sum], "8 bits, the sum in place")
    t = x.clone()
    same_bits([sgc.rms_norm(t, w, out=t).y], [sgc.rms_norm(x, w).y], "y in x without a residual")
    twice = sgc.rms_norm(x, w, residual=x)  # the same tensor as both
    equal_bits(twice.sum, lm8_ref.stream(x.cpu(), x.cpu()), "x + x")
    one = sgc.rms_norm_backward(dy, r.sum, w, r.rstd, dsum=ds)
    for at in ("dy", "s", "ds"):
        t = dict(dy=dy.clone(), s=r.sum.clone(), ds=ds.clone())
        got = sgc.rms_norm_backward(t["dy"], t["s"], w, r.rstd, dsum=t["ds"], dx=t[at])
        same_bits([t[at], got.dweight], [one.dx, one.dweight], f"dx in {at}")
    flat = torch.randn(cols, generator=g).cuda()
    was = flat.clone()
    got = sgc.rms_norm_backward(dy, r.sum, w, r.rstd, dweight=flat, accumulate=True, want_dx=False)
    assert got.dx is None and torch.equal(flat, was + one.dweight)


@DTYPES
@pytest.mark.parametrize("cols", [96, 130, 1000, 1031, 4096, 16384, 20000])
def test_the_stream_of_a_norm_in_place(cols, dtype):
    """y in x's place without a residual: the result's sum is what x was, as the backward pass needs it."""
    rows = 21
    g = gen(cols + 1)
    x, dy = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    w = torch.randn(cols, generator=g).cuda()
    announce(f"the stream of a norm in place, {rows}x{cols} {dtype}")
    apart = sgc.rms_norm(x.cuda(), w)
    for pad, offset in ((0, 0), (3, 1)):
        t, buf = rows_like(x, cols + pad, offset)
        got = sgc.rms_norm(t, w, out=t)
        assert got.y is t
        same_bits([got.y, got.rstd], [apart.y, apart.rstd], "y and rstd")
        equal_bits(got.sum, x, "sum")
        untouched(t, buf)
        b = sgc.rms_norm_backward(dy.cuda(), got.sum, w, got.rstd)
        (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, x, w, None, got.rstd, None)
        close(b.dx, dx, tdx, "dx", dtype)
        close(b.dweight, dw, tdw, "dweight")
    # a place for it given: there, x's own among them, which y may not take then
    t, s = x.cuda(), torch.empty(rows, cols, dtype=dtype, device="cuda")
    got = sgc.rms_norm(t, w, out=t, sum_out=s)
    assert got.sum is s
    equal_bits(s, x, "sum_out")
    t = x.cuda()
    got = sgc.rms_norm(t, w, sum_out=t)
    assert got.sum is t
    equal_bits(t, x, "the sum in x")
    same_bits([got.y], [apart.y], "y beside it")
    # apart, nothing is copied
    t = x.cuda()
    assert sgc.rms_norm(t, w).sum is t and sgc.rms_norm(t, w, out=s).sum is t and sgc.rms_norm_q8(t, w).sum is t


def test_the_stream_of_a_norm_in_place_captured():
    announce("the stream of a norm in place, captured")
    x = torch.randn(9, 1000, generator=gen(4)).to(BF16)
    u = x.cuda()
    sgc.rms_norm(u, out=u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sgc.rms_norm(u, out=u)
    for it in range(3):
        now = x * (1 + it)
        u.copy_(now)
        want = sgc.rms_norm(now.cuda())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same_bits([r.y, r.sum, r.rstd], [want.y, now.cuda(), want.rstd], f"replay {it}")


@DTYPES
@pytest.mark.parametrize("cols", [96, 650, 1031, 4096, 20000])
def test_rms_q8_with_the_sum_in_place(cols, dtype):
    """The sum in x's and in the residual's place beside 8 bits; the other one stays as it was."""
    rows = 41
    g = gen(cols + 2)
    x, res = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    w = torch.randn(cols, generator=g).cuda()
    announce(f"8 bits, the sum in place, {rows}x{cols} {dtype}")
    q = sgc.rms_norm_q8(x.cuda(), w, residual=res.cuda())
    for at in ("x", "res"):
        for pad, offset in ((0, 0), (3, 1)):
            t, buf = {}, {}
            for k, a in (("x", x), ("res", res)):
                t[k], buf[k] = rows_like(a, cols + pad, offset)
            got = sgc.rms_norm_q8(t["x"], w, residual=t["res"], sum_out=t[at])
            assert got.sum is t[at]
            same_bits([got.q8.q, got.q8.scale, got.sum, got.rstd], [q.q8.q, q.q8.scale, q.sum, q.rstd], f"sum in {at}")
            other = "res" if at == "x" else "x"
            equal_bits(t[other], x if other == "x" else res, f"{other} beside the sum in {at}")
            for k in t:
                untouched(t[k], buf[k])


def test_rms_edges():
    announce("rms edges")
    e = torch.empty(0, 10, device="cuda")
    r = sgc.rms_norm(e, residual=e)
    assert r.y.shape == (0, 10) and r.sum.shape == (0, 10)
    assert sgc.rms_norm_q8(e).q8.q.shape == (0, 10)
    flat = torch.full((10,), 3.0, device="cuda")
    sgc.rms_norm_backward(e, e, None, r.rstd, dweight=flat, accumulate=True)
    assert torch.equal(flat, torch.full_like(flat, 3.0))
    sgc.rms_norm_backward(e, e, None, r.rstd, dweight=flat)
    assert torch.equal(flat, torch.zeros_like(flat))
    for cols in (40, 300, 20000):
        x = torch.randn(9, cols, generator=gen(cols))
        x[1] = 0.0
        x[2, 7], x[3, 8], x[4, 9] = NAN, INF, -INF
        x[5] = 1e-44
        x[6] = 3e38
        x[7] *= 1e-20
        ok = [0, 1, 5, 7, 8]
        k = sgc.rms_norm(x.cuda(), eps=1e-6)
        (y, rstd), (ty, tr) = lm8_ref.rms(x[ok], None, 1e-6)
        close(k.y[ok], y, ty, "y beside broken rows")
        close(k.rstd[ok], rstd, tr, "rstd beside broken rows")
        assert torch.isnan(k.y[2]).all() and torch.isnan(k.y[3, 8]) and torch.isnan(k.y[4, 9])
        assert k.rstd[3] == 0 and k.rstd[6] == 0 and (k.y[6] == 0).all()
        q = sgc.rms_norm_q8(x.cuda(), eps=1e-6)
        want, (scale, _), (ts, _) = lm8_ref.rms_q8(x, None, 1e-6)
        equal_bits(q.q8.q, want, "q")
        close(q.q8.scale[ok], scale[ok], ts[ok] + 2.0 ** -148, "scale")
        assert torch.isnan(q.q8.scale[2:5]).all() and q.q8.scale[6] == 0 and q.q8.scale[1] == 0
        zero = sgc.rms_norm(torch.zeros(2, cols, device="cuda"), eps=0.0)  # 0 * inf, as the formula
        assert torch.isnan(zero.y).all()
        zero = sgc.rms_norm_q8(torch.zeros(2, cols, device="cuda"), eps=0.0)
        assert not zero.q8.q.any() and not zero.q8.scale.any()
    row = torch.randn(1, 300, generator=gen(1))
    r = sgc.rms_norm(row.cuda().expand(50, 300), residual=row.cuda().expand(50, 300))
    equal_bits(r.sum, (row + row).expand(50, 300), "one row for all")


# ------------------------------------------------------------------ 8 bits
Q_SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (70, 100), (33, 650), (4, 255), (9, 1024), (300, 1000), (7, 4099),
            (600, 1031), (3, 16384), (2, 16385), (2, 40001), (1, 131075), (2049, 64), (5000, 16)]
GROUPS = pytest.mark.parametrize("group", [0, 32, 64, 128, 256])


@DTYPES
@GROUPS
@pytest.mark.parametrize("rows,cols", Q_SHAPES, ids=str)
def test_quantize(rows, cols, group, dtype):
    x = stream_rows(rows, cols, dtype, gen(rows + cols))
    announce(f"quantize {rows}x{cols} group {group} {dtype}")
    c = sgc.quantize_q8(x.cuda(), group=group)
    q, scale = lm8_ref.quantize(x, group)
    equal_bits(c.q, q, "q")
    equal_bits(c.scale, scale, "scale")
    for to in (F32, dtype):
        equal_bits(sgc.dequantize_q8(c, to), lm8_ref.values(q, scale, group).to(to), f"values in {to}")


@DTYPES
@GROUPS
@pytest.mark.parametrize("offset,pad", [(0, 16), (1, 0), (3, 5), (8, 8)], ids=str)
@pytest.mark.parametrize("cols", [70, 650, 1024])
def test_quantize_strides_and_surroundings(dtype, group, offset, pad, cols):
    rows = 41
    x = stream_rows(rows, cols, dtype, gen(cols))
    announce(f"quantize strides {dtype} group {group} cols {cols} offset {offset} pad {pad}")
    xd = rows_like(x, cols + pad, offset)[0]
    qd, qbuf = rows_like(torch.zeros(rows, cols, dtype=torch.int8), cols + pad + 1, offset + 2)
    q, scale = lm8_ref.quantize(x, group)
    sc, sbuf = rows_like(torch.zeros_like(scale), offset=1)
    c = sgc.quantize_q8(xd, group=group, out=sgc.Quantized(qd, sc, group))
    equal_bits(c.q, q, "q")
    equal_bits(c.scale, scale, "scale")
    untouched(qd, qbuf)
    untouched(sc, sbuf)
    v, vbuf = rows_like(x * 0, cols + pad, offset + 1)
    sgc.dequantize_q8(c, dtype, out=v)
    equal_bits(v, lm8_ref.values(q, scale, group).to(dtype), "values")
    untouched(v, vbuf)


@GROUPS
@DTYPES
def test_quantize_edges(group, dtype):
    announce(f"quantize edges group {group} {dtype}")
    assert sgc.quantize_q8(torch.empty(0, 40, device="cuda", dtype=dtype), group=group).q.shape == (0, 40)
    f = torch.finfo(dtype)
    for cols in (300, 20000):
        x = torch.randn(8, cols, generator=gen(1)).to(dtype)
        x[1, ::3], x[2, 5], x[3, 70], x[4, 290] = 0.0, NAN, INF, -INF
        x[5, :64] = 0.0
        x[6, 64:128] = f.smallest_normal * f.eps  # the smallest number there is
        x[7, 10], x[7, 100] = f.max, f.min
        c = sgc.quantize_q8(x.cuda(), group=group)
        q, scale = lm8_ref.quantize(x, group)
        equal_bits(c.q, q, "q")
        equal_bits(c.scale, scale, "scale")
        equal_bits(sgc.dequantize_q8(c, dtype), lm8_ref.values(q, scale, group).to(dtype), "values")
    c = sgc.quantize_q8(x[:1].cuda().expand(9, cols), group=group)  # one row for all
    equal_bits(c.q, q[:1].expand(9, cols), "one row for all")


# ---------------------------------------- norms from activations in 8 bits
def stats_of(v, kind):
    v = v.double()
    mean = v.mean(1)
    if kind == "rms":
        return None, (v.square().mean(1) + 1e-6).rsqrt().float()
    return mean.float(), (v.var(1, unbiased=False) + 1e-6).rsqrt().float()


def backward_q8(kind, dy, c, w, b, mean, rstd, **kw):
    if kind == "rms":
        return sgc.rms_norm_backward_q8(dy, c, w, rstd, **kw)
    return sgc.layer_norm_backward_q8(dy, c, w, b, mean, rstd, **kw)


def check_backward_q8(kind, rows, cols, group, dtype, dsum=True):
    g = gen(rows * 3 + cols)
    x = stream_rows(rows, cols, dtype, g)
    q, scale = lm8_ref.quantize(x, group)
    v = lm8_ref.values(q, scale, group)
    mean, rstd = stats_of(v, kind)
    dy, ds = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    ds = ds if dsum else None
    b = b if kind == "layer" else None
    cuda = lambda t: None if t is None else t.cuda()
    r = backward_q8(kind, dy.cuda(), sgc.Quantized(q.cuda(), scale.cuda(), group), w.cuda(), cuda(b), cuda(mean),
                    rstd.cuda(), dsum=cuda(ds), want_y=True)
    (dx, dw, db), (tdx, tdw, tdb) = lm8_ref.backward(dy, v, w, mean, rstd, ds)
    close(r.dx, dx, tdx, "dx", dtype)
    close(r.dweight, dw, tdw, "dweight")
    if kind == "layer":
        close(r.dbias, db, tdb, "dbias")
    else:
        assert r.dbias is None
    y, ty = lm8_ref.normed(v, w, b, mean, rstd)
    close(r.y, y, ty, "y", dtype)


@DTYPES
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("rows,cols", SHAPES, ids=str)
def test_norm_backward_from_8_bits(rows, cols, kind, dtype):
    group = (32, 64, 128, 256, 0)[(rows + cols) % 5]
    announce(f"{kind} backward from 8 bits {rows}x{cols} group {group} {dtype}")
    check_backward_q8(kind, rows, cols, group, dtype, dsum=cols % 2 == 0)


@GROUPS
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [70, 650, 1027, 8200])
def test_norm_backward_from_8_bits_groups(cols, kind, group):
    announce(f"{kind} backward from 8 bits, group {group}, {cols} columns")
    for dtype in (F32, BF16):
        check_backward_q8(kind, 45, cols, group, dtype)


@DTYPES
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("offset,pad", [(0, 16), (1, 0), (3, 5), (4, 12)], ids=str)
@pytest.mark.parametrize("cols,weight", [(100, "same"), (650, "fp32"), (1031, "none"), (20003, "same")], ids=str)
def test_norm_backward_from_8_bits_strides(dtype, kind, offset, pad, cols, weight):
    rows, group = 37, 64
    g = gen(offset + cols)
    announce(f"{kind} backward from 8 bits strides {dtype} cols {cols} offset {offset} pad {pad} weight {weight}")
    q, scale = lm8_ref.quantize(stream_rows(rows, cols, dtype, g), group)
    v = lm8_ref.values(q, scale, group)
    mean, rstd = stats_of(v, kind)
    dy, ds = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    wt = dtype if weight == "same" else F32
    w = None if weight == "none" else torch.randn(cols, generator=g).to(wt)
    b = torch.randn(cols, generator=g).to(wt) if kind == "layer" and weight != "none" else None
    at = lambda t, k: None if t is None else rows_like(t[None], offset=k)[0][0]
    c = sgc.Quantized(rows_like(q, cols + pad, offset)[0], rows_like(scale, offset=1)[0], group)
    dyd, dsd = rows_like(dy, cols + pad + 1, offset + 1)[0], rows_like(ds, cols + 2, 3)[0]
    dxd, dxbuf = rows_like(dy * 0, cols + pad, offset)
    yd, ybuf = rows_like(dy * 0, cols + 2 * pad, 8 - offset)
    flat = torch.full((2 * cols + 5,), 7.0, device="cuda")
    kw = dict(dbias=flat[cols + 2:2 * cols + 2]) if kind == "layer" else {}
    r = backward_q8(kind, dyd, c, at(w, 1), at(b, 3), at(mean, 1), at(rstd, 1), dsum=dsd, dx=dxd, y=yd,
                    dweight=flat[1:1 + cols], **kw)
    (dx, dw, db), (tdx, tdw, tdb) = lm8_ref.backward(dy, v, w, mean, rstd, ds)
    close(r.dx, dx, tdx, "dx", dtype)
    close(r.dweight, dw, tdw, "dweight")
    if kind == "layer":
        close(r.dbias, db, tdb, "dbias")
    y, ty = lm8_ref.normed(v, w, b, mean, rstd)
    close(r.y, y, ty, "y", dtype)
    untouched(dxd, dxbuf)
    untouched(yd, ybuf)
    assert [float(flat[k]) for k in (0, cols + 1, 2 * cols + 2, 2 * cols + 4)] == [7.0] * 4


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [100, 1000, 20000])
def test_norm_backward_from_8_bits_wants(kind, cols):
    """Each output alone, in place, added, and no rows at all."""
    announce(f"{kind} backward from 8 bits, outputs alone, {cols} columns")
    rows, g = 50, gen(cols)
    x = stream_rows(rows, cols, BF16, g).cuda()
    c = sgc.quantize_q8(x, group=128)
    mean, rstd = [None if t is None else t.cuda() for t in stats_of(x.cpu(), kind)]
    dy, ds = [torch.randn(rows, cols, generator=g).to(BF16).cuda() for _ in range(2)]
    w = torch.randn(cols, generator=g).cuda()
    b = w.flip(0).contiguous() if kind == "layer" else None
    call = lambda dy=dy, ds=ds, **kw: backward_q8(kind, dy, c, w, b, mean, rstd, dsum=ds, **kw)
    one = call(want_y=True)
    alone = call(want_dx=False, want_y=True)
    assert alone.dx is None
    same_bits([alone.dweight, alone.dbias, alone.y], [one.dweight, one.dbias, one.y], "without dx")
    alone = call()
    assert alone.y is None
    same_bits([alone.dx, alone.dweight], [one.dx, one.dweight], "without y")
    t = dy.clone()
    same_bits([call(dy=t, dx=t, want_y=True).dx, t], [one.dx, one.dx], "dx in dy")
    t = ds.clone()
    same_bits([call(ds=t, dx=t).dx, t], [one.dx, one.dx], "dx in dsum")
    flat = torch.ones(2 * cols, device="cuda")
    kw = dict(dbias=flat[cols:]) if kind == "layer" else {}
    call(dweight=flat[:cols], accumulate=True, **kw)
    assert torch.equal(flat[:cols], 1 + one.dweight)
    if kind == "layer":
        assert torch.equal(flat[cols:], 1 + one.dbias)
    none = sgc.Quantized(c.q[:0], c.scale[:0], 128)
    r = backward_q8(kind, dy[:0], none, w, b, None if mean is None else mean[:0], rstd[:0], want_y=True)
    assert r.dx.shape == (0, cols) and r.y.shape == (0, cols) and not r.dweight.any()


@pytest.mark.parametrize("cols", [100, 650, 4099, 9000, 20000])
def test_layer_norm_from_8_bits_with_a_weight_or_a_bias_alone(cols):
    """The one that is not given counts as 1 or 0, in the gradients and in y."""
    rows, group = 19, 128
    g = gen(cols + 3)
    announce(f"layer norm from 8 bits, weight or bias alone, {cols} columns")
    for dtype in (F32, BF16):
        q, scale = lm8_ref.quantize(stream_rows(rows, cols, dtype, g), group)
        v = lm8_ref.values(q, scale, group)
        mean, rstd = stats_of(v, "layer")
        dy = torch.randn(rows, cols, generator=g).to(dtype)
        p = torch.randn(cols, generator=g)
        for pt in (F32, dtype):
            for w, b in ((p.to(pt), None), (None, p.to(pt))):
                cuda = lambda t: None if t is None else t.cuda()
                r = sgc.layer_norm_backward_q8(dy.cuda(), sgc.Quantized(q.cuda(), scale.cuda(), group), cuda(w),
                                               cuda(b), mean.cuda(), rstd.cuda(), want_y=True)
                (dx, dw, db), (tdx, tdw, tdb) = lm8_ref.backward(dy, v, w, mean, rstd, None)
                close(r.dx, dx, tdx, "dx", dtype)
                close(r.dweight, dw, tdw, "dweight")
                close(r.dbias, db, tdb, "dbias")
                y, ty = lm8_ref.normed(v, w, b, mean, rstd)
                close(r.y, y, ty, "y", dtype)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("cols", [100, 650, 4096, 20000])
def test_a_broken_group_stays_in_its_row_and_columns(cols, kind):
    """A group whose scale is NaN: its row's dx, its columns' dweight and its own y are NaN, all else as without it."""
    rows, group, at = 25, 32, 7
    g = gen(cols + 4)
    announce(f"{kind} backward from 8 bits, a broken group, {cols} columns")
    x = stream_rows(rows, cols, BF16, g)
    q, scale = lm8_ref.quantize(x, group)
    mean, rstd = [None if t is None else t.cuda() for t in stats_of(lm8_ref.values(q, scale, group), kind)]
    dy, w = torch.randn(rows, cols, generator=g).to(BF16).cuda(), torch.randn(cols, generator=g).cuda()
    call = lambda s: backward_q8(kind, dy, sgc.Quantized(q.cuda(), s.cuda(), group), w,
                                 w.flip(0).contiguous() if kind == "layer" else None, mean, rstd, want_y=True)
    one = call(scale)
    broken = scale.clone()
    broken[at, 1] = NAN
    r = call(broken)
    rest = [k for k in range(rows) if k != at]
    outside = torch.ones(cols, dtype=torch.bool)
    outside[group:2 * group] = False
    same_bits([r.dx[rest], r.y[rest], r.y[at][outside], r.dweight[outside], r.dbias],
              [one.dx[rest], one.y[rest], one.y[at][outside], one.dweight[outside], one.dbias], "beside the group")
    for t in (r.dx[at], r.y[at][~outside], r.dweight[~outside]):
        assert torch.isnan(t).all()


def test_checkpoint_gradient_against_differences():
    """The gradient at the values that the 8 bits stand for, in fp32, against differences of the norm's formula."""
    announce("gradient from 8 bits against differences")
    rows, cols = 3, 40
    g = gen(11)
    for kind in ("rms", "layer"):
        c = sgc.quantize_q8(torch.randn(rows, cols, generator=g).cuda(), group=32)
        v = sgc.dequantize_q8(c).cpu().double()
        w, b, dy = [torch.randn(*s, generator=g).double() for s in ((cols,), (cols,), (rows, cols))]
        mean, rstd = stats_of(v, kind)

        def loss(v):
            y = lm8_ref.rms(v, w, 1e-6)[0][0] if kind == "rms" else lm_ref.norm(v, w, b, 1e-6)[0][0]
            return (y * dy).sum(1)

        f = lambda t: t.float().cuda()
        r = backward_q8(kind, f(dy), c, f(w), f(b) if kind == "layer" else None, None if mean is None else mean.cuda(),
                        rstd.cuda())
        step, want = 1e-4, torch.zeros(rows, cols, dtype=torch.float64)
        for k in range(cols):
            d = torch.zeros(cols, dtype=torch.float64)
            d[k] = step
            want[:, k] = (loss(v + d) - loss(v - d)) / (2 * step)
        # differences are off by step^2 / 6 of a third derivative, a few tens here; fp32 by some 1e-6 of the terms
        assert float((r.dx.cpu().double() - want).abs().max()) < 1e-5


# ---------------------------------------------------------------- products
def whole(rows, width, seed, low=-127):
    return torch.randint(low, 128, (rows, width), generator=gen(seed), dtype=torch.int32).to(torch.int8)


def check_product(xq, wq, bias, dtype, xd=None, wd=None, out=None, seed=0):
    g = gen(seed + 5)
    xs, ws = torch.rand(len(xq), 1, generator=g) * 0.02, torch.rand(len(wq), 1, generator=g) * 0.02
    b = torch.randn(len(wq), generator=g) * 5 if bias else None
    y = sgc.int8_linear(sgc.Quantized(xq.cuda() if xd is None else xd, xs.cuda()),
                        sgc.Quantized(wq.cuda() if wd is None else wd, ws.cuda()), None if b is None else b.cuda(),
                        dtype=dtype, out=out)
    ref, tol = lm8_ref.product(xq, xs, wq, ws, b)
    close(y, ref, tol, "y", dtype)


P_SHAPES = [(1, 1, 1), (1, 16, 1), (2, 17, 3), (1, 64, 50), (1, 1024, 5000), (3, 650, 1001), (4, 4096, 260),
            (5, 15, 700), (8, 1024, 98), (16, 128, 16), (16, 512, 1000), (17, 512, 1000), (31, 100, 33),
            (32, 4096, 1024), (33, 2048, 257), (63, 640, 64), (64, 64, 64), (65, 127, 129), (100, 650, 10000),
            (127, 128, 128), (128, 1024, 512), (129, 129, 131), (255, 256, 300), (256, 256, 256), (257, 513, 255),
            (300, 96, 2000), (512, 512, 513), (777, 650, 1001), (1000, 64, 3), (2049, 1040, 98), (40, 16384, 100),
            (2, 16385, 40), (260, 33000, 270)]


@DTYPES
@pytest.mark.parametrize("rows,width,out", P_SHAPES, ids=str)
def test_product(rows, width, out, dtype):
    announce(f"product {rows}x{width}x{out} {dtype}")
    check_product(whole(rows, width, rows), whole(out, width, out + 1), bool(width % 2 or out % 2), dtype, seed=rows)


@pytest.mark.parametrize("rows", [1, 5, 16, 30, 70, 150, 300, 520])
@pytest.mark.parametrize("width", [48, 650, 1000])
@pytest.mark.parametrize("xo,xp,wo,wp", [(0, 16, 0, 16), (16, 0, 32, 48), (1, 0, 0, 0), (0, 0, 3, 5), (5, 3, 9, 1),
                                         (8, 8, 4, 4)], ids=str)
def test_product_strides(rows, width, xo, xp, wo, wp):
    """Rows at every alignment: their neighbours hold what would show if it were read."""
    out = 333
    announce(f"product strides {rows}x{width}x{out} at {xo} {xp} {wo} {wp}")
    xq, wq = whole(rows, width, 1), whole(out, width, 2)
    up = lambda p: p if p % 16 else -(-width // 16) * 16 - width + p
    xd, wd = rows_like(xq, width + up(xp), xo, 101)[0], rows_like(wq, width + up(wp), wo, 103)[0]
    y, buf = rows_like(torch.zeros(rows, out), out + 3, 1)
    check_product(xq, wq, True, F32, xd, wd, y)
    untouched(y, buf)
    y, buf = rows_like(torch.zeros(rows, out, dtype=BF16), out + 5, 3)
    check_product(xq, wq, False, BF16, xd, wd, y)
    untouched(y, buf)


@pytest.mark.parametrize("rows,width,out", [(3700, 130, 4001), (3600, 128, 4090), (3599, 17, 3841), (700, 1100, 6001),
                                            (690, 1152, 6000), (1000, 650, 2001), (1001, 1024, 2048),
                                            (130, 1500, 1031), (257, 4000, 129)], ids=str)
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
@DTYPES
def test_product_of_every_tile(rows, width, out, aligned, dtype):
    """Sizes that take the tiles of 256, 128 and 64 (in four and in eight steps), each with ragged edges."""
    announce(f"product {rows}x{width}x{out} aligned {aligned} {dtype}")
    xq, wq = whole(rows, width, 1), whole(out, width, 2)
    up = -(-width // 16) * 16 + (0 if aligned else 3)
    xd, wd = rows_like(xq, up, 0, 101)[0], rows_like(wq, up, 0 if aligned else 5, 103)[0]
    y, buf = rows_like(torch.zeros(rows, out, dtype=dtype), out + 1, 1)
    check_product(xq, wq, True, dtype, xd, wd, y)
    untouched(y, buf)


@pytest.mark.parametrize("rows,out", [(1, 40), (20, 40), (130, 200), (300, 300)], ids=str)
def test_product_at_the_largest_sums(rows, out):
    """-128 times -128, 131071 times: 2^31 less 2^14."""
    width = (1 << 17) - 1
    announce(f"largest sums {rows}x{width}x{out}")
    x = torch.full((rows, width), -128, dtype=torch.int8, device="cuda")
    w = torch.full((out, width), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = lambda n: torch.ones(n, 1, device="cuda")
    y = sgc.int8_linear(sgc.Quantized(x, one(rows)), sgc.Quantized(w, one(out)), dtype=F32)
    want = torch.full((rows, out), float(torch.tensor(128 * 128 * width).float()))
    want[:, 1] = float(torch.tensor(-128 * 127 * width).float())
    equal_bits(y, want, "y")


def test_product_edges():
    announce("product edges")
    w = sgc.quantize_q8(torch.randn(30, 70, generator=gen(1)).cuda(), group=0)
    e = sgc.quantize_q8(torch.empty(0, 70, device="cuda"), group=0)
    assert sgc.int8_linear(e, w).shape == (0, 30)
    x = torch.randn(6, 70, generator=gen(2))
    x[1], x[2, 3], x[4, 5] = 0.0, NAN, INF
    for rows in (6, 60, 300):  # every kernel
        c = sgc.quantize_q8(x.repeat(rows // 6, 1).cuda(), group=0)
        y = sgc.int8_linear(c, w, dtype=F32).view(rows // 6, 6, 30)
        assert (y[:, 1] == 0).all() and torch.isnan(y[:, 2]).all() and torch.isnan(y[:, 4]).all()
        ref, tol = lm8_ref.product(c.q[[0, 3, 5]], c.scale[[0, 3, 5]], w.q, w.scale, None)
        close(y[-1][[0, 3, 5]], ref, tol, "rows beside broken ones")
    one = sgc.int8_linear(sgc.Quantized(c.q[:1].expand(40, 70), c.scale[:1].expand(40, 1).contiguous()), w, dtype=F32)
    same_bits([one], [y[0, :1].expand(40, 30)], "one row for all")
    one = sgc.int8_linear(c, sgc.Quantized(w.q[:1].expand(40, 70), w.scale[:1].expand(40, 1).contiguous()), dtype=F32)
    same_bits([one], [y.view(300, 30)[:, :1].expand(300, 40)], "one channel for all")


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_product_past_32_bits(rows):
    """Rows of x, of the weights and of y that lie past 2^31 and 2^32 bytes."""
    announce(f"product past 32 bits, {rows} rows")
    width, out, far = 272, 70, (1 << 32) + 4096
    xq, wq = whole(rows, width, 3), whole(out, width, 4)
    buf = torch.zeros(far + 4096, dtype=torch.int8, device="cuda")
    step = far // (out - 1) // 16 * 16
    wd = buf.as_strided((out, width), (step, 1))
    wd.copy_(wq)
    check_product(xq, wq, True, F32, None, wd)
    step = far // (rows - 1) // 16 * 16
    xd = buf.as_strided((rows, width), (step, 1))
    xd.copy_(xq)
    ybuf = torch.zeros((1 << 31) + 4096, dtype=F32, device="cuda")
    y = ybuf.as_strided((rows, out), ((1 << 31) // (rows - 1), 1))
    check_product(xq, wq, False, F32, xd, None, y)


@pytest.mark.parametrize("rows,width,out", [(1, 1024, 50000), (32, 4096, 4096), (2000, 4096, 10000)], ids=str)
def test_product_large(rows, width, out):
    """Against integer sums of some rows and channels."""
    announce(f"product {rows}x{width}x{out}")
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (rows, width), device="cuda", generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (out, width), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.rand(rows, 1, device="cuda", generator=g), torch.rand(out, 1, device="cuda", generator=g)
    y = sgc.int8_linear(sgc.Quantized(xq, xs), sgc.Quantized(wq, ws), dtype=F32)
    ref, tol = lm8_ref.product(xq, xs, wq, ws, None)
    close(y, ref, tol, "y")


# --------------------------------------------------------- as they are used
def step_tensors(rows=48, cols=640, vocab=1000):
    g = gen(rows)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    return dict(x=r(rows, cols).to(BF16), res=r(rows, cols).to(BF16), w=r(cols), b=r(cols), head=r(vocab, cols),
                dy=r(rows, cols).to(BF16), ds=r(rows, cols).to(BF16), bias=r(vocab))


def all_calls(t, ws=None, stream=None):
    """Every call of the set, one after the other on one stream."""
    kw = dict(stream=stream)
    ws = ws or [None] * 3
    head = sgc.quantize_q8(t["head"], group=0, **kw)
    n = sgc.rms_norm_q8(t["x"], t["w"], residual=t["res"], **kw)
    z = sgc.int8_linear(n.q8, head, t["bias"], **kw)
    y = sgc.rms_norm(t["x"], t["w"], residual=t["res"], **kw)
    b = sgc.rms_norm_backward(t["dy"], y.sum, t["w"], y.rstd, dsum=t["ds"], ws=ws[0], **kw)
    c = sgc.quantize_q8(y.sum, group=64, **kw)
    v = sgc.dequantize_q8(c, BF16, **kw)
    rb = sgc.rms_norm_backward_q8(t["dy"], c, t["w"], y.rstd, dsum=t["ds"], want_y=True, ws=ws[1], **kw)
    ln = sgc.layer_norm(v, t["w"], t["b"], **kw)
    lb = sgc.layer_norm_backward_q8(t["dy"], c, t["w"], t["b"], ln.mean, ln.rstd, want_y=True, ws=ws[2], **kw)
    return [head.q, head.scale, n.q8.q, n.q8.scale, n.sum, z, y.y, y.rstd, b.dx, b.dweight, c.q, c.scale, v, rb.dx,
            rb.dweight, rb.y, lb.dx, lb.dweight, lb.dbias, lb.y]


def workspaces(rows, cols, fill):
    sizes = [sgc.rms_norm_backward_workspace_bytes(rows, cols, BF16),
             sgc.norm_backward_q8_workspace_bytes(rows, cols, group=64, dtype=BF16),
             sgc.norm_backward_q8_workspace_bytes(rows, cols, kind=sgc.NORM_LAYER, group=64, dtype=BF16)]
    return [torch.full((n,), fill, dtype=torch.uint8, device="cuda") for n in sizes]


@pytest.mark.parametrize("rows,cols,vocab", [(48, 640, 1000), (1, 1024, 5000), (500, 98, 130), (3, 20000, 64)], ids=str)
def test_same_bits_whatever_the_workspace_held(rows, cols, vocab):
    announce(f"same bits {rows}x{cols}x{vocab}")
    t = step_tensors(rows, cols, vocab)
    first = all_calls(t)
    for fill in (0, 0x5A, 0xFF):
        same_bits(all_calls(t, ws=workspaces(rows, cols, fill)), first, f"workspace of {fill}")


def test_streams():
    announce("streams")
    t = step_tensors()
    first = all_calls(t)
    s = torch.cuda.Stream()
    u = {k: torch.empty_like(v) for k, v in t.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for k in t:
            u[k].copy_(t[k])  # the calls have to wait for this: same stream
    other = all_calls(u, stream=s)
    s.synchronize()
    same_bits(other, first, "another stream")


@pytest.mark.parametrize("rows,cols,vocab", [(48, 640, 1000), (1, 1024, 5000), (300, 650, 300)], ids=str)
def test_graph_replays(rows, cols, vocab):
    announce(f"graph {rows}x{cols}x{vocab}")
    t = step_tensors(rows, cols, vocab)
    u = {k: v.clone() for k, v in t.items()}
    ws = workspaces(rows, cols, 0)
    all_calls(u, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(u, ws=ws)
    torch.cuda.synchronize()
    for it in range(4):
        for k in ("x", "dy", "head"):
            u[k].copy_(torch.roll(t[k], it, 1) * (1 + it))
        want = all_calls(u)  # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same_bits(out, want, f"replay {it}")


def test_captured_call_needs_its_own_workspace():
    announce("a captured backward call without a workspace is refused")
    t = step_tensors()
    y = sgc.rms_norm(t["x"], t["w"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="workspace"):
        with torch.cuda.graph(graph):
            t["dy"].clone()
            sgc.rms_norm_backward(t["dy"], y.sum, t["w"], y.rstd)
    torch.cuda.synchronize()


def test_teacher_in_8_bits_teaches_a_student():
    """Norm, product, the teacher's list, the student's loss and gradient, its norm's backward pass from 8 bits."""
    announce("teacher in 8 bits")
    rows, cols, vocab = 64, 512, 1003
    t = step_tensors(rows, cols, vocab)
    head = sgc.quantize_q8(t["head"] * cols ** -0.5, group=0)
    n = sgc.rms_norm_q8(t["x"], t["w"], residual=t["res"])
    z = sgc.int8_linear(n.q8, head, dtype=F32)
    ref, tol = lm8_ref.product(n.q8.q, n.q8.scale, head.q, head.scale, None)
    close(z, ref, tol, "the teacher's logits")
    top = sgc.token_logprobs(z, top=16)
    s = sgc.rms_norm(t["x"], t["w"])
    kept = sgc.quantize_q8(s.sum, group=128)
    logits = s.y @ t["head"].to(BF16).t()
    d = sgc.distill(logits, top.top_idx, top.top_logp, mode=sgc.DISTILL_TAIL,
                    dloss=torch.full((rows,), 1.0 / rows, device="cuda"))
    dy = d.dlogits @ t["head"].to(BF16)
    flat = torch.zeros(cols, device="cuda")
    b = sgc.rms_norm_backward_q8(dy, kept, t["w"], s.rstd, dweight=flat, want_y=True)
    v = lm8_ref.values(kept.q, kept.scale, 128)
    (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, v, t["w"], None, s.rstd, None)
    close(b.dx, dx, tdx, "dx", BF16)
    close(flat, dw, tdw, "dweight")
    # the activations given again differ from the forward pass' by half a step of their group, not more
    half = kept.scale.repeat_interleave(128, 1) / 2 * s.rstd[:, None] * t["w"].abs()
    off = (b.y.float() - s.y.float()).abs()
    assert bool((off <= half * 1.001 + 2 * 2.0 ** -8 * s.y.float().abs() + half * 2.0 ** -7).all())


@pytest.mark.parametrize("name", ["sum_out", "out", "dx", "dweight", "q", "scale", "values", "y", "product"])
def test_a_write_into_what_autograd_saved_is_noticed(name):
    announce(f"in place over a saved tensor: {name}")
    x = torch.randn(6, 40, device="cuda")
    v = torch.ones(6, device="cuda")
    c, h = sgc.quantize_q8(x, group=32), sgc.quantize_q8(x[:, :40], group=0)
    calls = {
        "sum_out": lambda t: sgc.rms_norm(x, residual=x, sum_out=t), "out": lambda t: sgc.rms_norm(x, out=t),
        "dx": lambda t: sgc.rms_norm_backward(x, x, None, v, dx=t),
        "dweight": lambda t: sgc.rms_norm_backward(x, x, None, v, dweight=t.view(-1)[:40]),
        "q": lambda t: sgc.quantize_q8(x, out=sgc.Quantized(t.view(torch.int8)[:, :40], c.scale, 32), group=32),
        "scale": lambda t: sgc.quantize_q8(x, out=sgc.Quantized(c.q, t.view(-1)[:12].view(6, 2), 32), group=32),
        "values": lambda t: sgc.dequantize_q8(c, out=t), "y": lambda t: sgc.rms_norm_backward_q8(x, c, None, v, y=t),
        "product": lambda t: sgc.int8_linear(h, h, dtype=F32, out=t.view(-1)[:36].view(6, 6)),
    }
    leaf = torch.zeros(6, 40, device="cuda", requires_grad=True)
    saved = leaf.exp()
    calls[name](saved.detach())
    with pytest.raises(RuntimeError, match="inplace operation"):
        saved.sum().backward()


# ------------------------------------------------- large calls, many rows
@pytest.mark.parametrize("cols,dtype", [(98, BF16), (650, F32), (1000, F16), (2048, BF16), (4099, BF16), (8192, F16),
                                        (16384, F32)], ids=str)
def test_large_norms(cols, dtype):
    """So many rows that a call moves more than the last-level cache holds: some rows, and the sums over all."""
    rows = (256 << 20) // (2 * cols * dtype.itemsize) + 3
    announce(f"large norms {rows}x{cols} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    mk = lambda: torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(generator=g)
    x, res, dy, ds = mk(), mk(), mk(), mk()
    w = torch.empty(cols, device="cuda").normal_(generator=g)
    pick = torch.tensor([0, 1, 2, 3, rows // 2, rows - 2, rows - 1])
    r = sgc.rms_norm(x, w, residual=res)
    s = lm8_ref.stream(x[pick].cpu(), res[pick].cpu())
    equal_bits(r.sum[pick], s, "sum")
    (y, rstd), (ty, tr) = lm8_ref.rms(s, w, 1e-6)
    close(r.y[pick], y, ty, "y", dtype)
    q = sgc.rms_norm_q8(x, w, residual=res)
    same_bits([q.sum, q.rstd], [r.sum, r.rstd], "8 bits beside y")
    equal_bits(q.q8.q[pick], lm8_ref.rms_q8(s, w, 1e-6)[0], "q")
    b = sgc.rms_norm_backward(dy, r.sum, w, r.rstd, dsum=ds)
    (dx, _, _), (tdx, _, _) = lm8_ref.backward(dy[pick], s, w, None, r.rstd[pick], ds[pick])
    close(b.dx[pick], dx, tdx, "dx", dtype)
    dw = torch.zeros(cols, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(dw)
    c = sgc.quantize_q8(r.sum, group=64)
    want, scale = lm8_ref.quantize(s, 64)
    equal_bits(c.q[pick], want, "8 bits")
    equal_bits(c.scale[pick], scale, "their scales")
    v = sgc.dequantize_q8(c, dtype)
    equal_bits(v[pick], lm8_ref.values(want, scale, 64).to(dtype), "values")
    k = sgc.rms_norm_backward_q8(dy, c, w, r.rstd, dsum=ds, want_y=True)
    (dx, _, _), (tdx, _, _) = lm8_ref.backward(dy[pick], lm8_ref.values(want, scale, 64), w, None, r.rstd[pick],
                                               ds[pick])
    close(k.dx[pick], dx, tdx, "dx from 8 bits", dtype)
    dw8, mag8 = torch.zeros_like(dw), torch.zeros_like(dw)
    for a in range(0, rows, 4096):
        part = slice(a, a + 4096)
        for to, m, at in ((dw, mag, r.sum[part].double()), (dw8, mag8, sgc.dequantize_q8(
                sgc.Quantized(c.q[part], c.scale[part].contiguous(), 64)).double())):
            t = dy[part].double() * at * r.rstd[part].double()[:, None]
            to += t.sum(0)
            m += t.abs().sum(0)
    tol = (64 + rows // 64 + 2) * lm_ref.U
    close(b.dweight, dw.cpu(), tol * mag.cpu(), "dweight")
    close(k.dweight, dw8.cpu(), tol * mag8.cpu(), "dweight from 8 bits")


def test_rows_past_32_bits():
    """Rows more than 2^31 elements, and 2^32 bytes, apart."""
    announce("rows past 32 bits")
    rows, cols, step = 3, 1003, (1 << 31) + 72
    g = gen(9)
    x, dy = [torch.randn(rows, cols, generator=g).to(BF16) for _ in range(2)]
    w = torch.randn(cols, generator=g)
    far = [torch.empty((rows - 1) * step + cols, dtype=BF16, device="cuda").as_strided((rows, cols), (step, 1))
           for _ in range(3)]
    q = torch.empty((rows - 1) * 2 * step + cols, dtype=torch.int8, device="cuda").as_strided((rows, cols),
                                                                                           (2 * step, 1))
    xd, yd, dxd = far
    xd.copy_(x)
    r = sgc.rms_norm(xd, w.cuda(), out=yd)
    (y, rstd), (ty, tr) = lm8_ref.rms(x, w, 1e-6)
    close(r.y, y, ty, "y", BF16)
    for group in (0, 64):
        want, scale = lm8_ref.quantize(x, group)
        c = sgc.quantize_q8(xd, group=group,
                            out=sgc.Quantized(q, torch.empty(scale.shape, device="cuda"), group))
        equal_bits(c.q, want, "q")
        equal_bits(c.scale, scale, "scale")
        equal_bits(sgc.dequantize_q8(c, BF16, out=yd), lm8_ref.values(want, scale, group).to(BF16), "values")
        b = sgc.rms_norm_backward_q8(dy.cuda(), c, w.cuda(), r.rstd, dx=dxd, y=yd)
        v = lm8_ref.values(want, scale, group)
        (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, v, w, None, r.rstd, None)
        close(b.dx, dx, tdx, "dx from 8 bits", BF16)
        close(b.dweight, dw, tdw, "dweight from 8 bits")
    b = sgc.rms_norm_backward(dy.cuda(), xd, w.cuda(), r.rstd, dx=dxd)
    (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, x, w, None, r.rstd, None)
    close(b.dx, dx, tdx, "dx", BF16)
    close(b.dweight, dw, tdw, "dweight")


def test_two_streams_at_once():
    """The same calls on two streams that run side by side, each with its own cached workspaces."""
    announce("two streams at once")
    t, u = step_tensors(300, 640, 1000), step_tensors(301, 640, 1000)
    want = [all_calls(t), all_calls(u)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for k, (s, v) in enumerate(((a, t), (b, u))):
            got.append((k, all_calls(v, stream=s)))
    torch.cuda.synchronize()
    for k, r in got:
        same_bits(r, want[k], f"stream {k}")


def test_binding_refuses_mismatches():
    announce("mismatched calls are refused")
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    w, v = torch.zeros(64, device="cuda"), torch.zeros(4, device="cuda")
    c, k = sgc.quantize_q8(x, group=32), sgc.quantize_q8(x, group=0)
    short = sgc.Quantized(k.q[:, :32], k.scale)
    for f in (lambda: sgc.rms_norm(x, residual=x[:, :32]), lambda: sgc.rms_norm(x, residual=x.float()),
              lambda: sgc.rms_norm(x, w[:32]), lambda: sgc.rms_norm(x, w.half()), lambda: sgc.rms_norm(x, out=x[:2]),
              lambda: sgc.rms_norm(x.t()), lambda: sgc.rms_norm(x, sum_out=x.float()),
              lambda: sgc.rms_norm_q8(x, out=c), lambda: sgc.rms_norm_q8(x, out=short),
              lambda: sgc.rms_norm_backward(x, x[:, :32], None, v), lambda: sgc.rms_norm_backward(x, x, None, v[:3]),
              lambda: sgc.rms_norm_backward(x, x, None, v, dsum=x.float()),
              lambda: sgc.rms_norm_backward(x, x, None, v, accumulate=True),
              lambda: sgc.rms_norm_backward(x, x, None, v, dweight=w[:32]),
              lambda: sgc.quantize_q8(x, group=48), lambda: sgc.quantize_q8(x, group=64, out=c),
              lambda: sgc.quantize_q8(x, group=0, out=short), lambda: sgc.dequantize_q8(c, torch.float64),
              lambda: sgc.dequantize_q8(c, BF16, out=x[:2]),
              lambda: sgc.dequantize_q8(sgc.Quantized(c.q, c.scale[:, :1], 32)),
              lambda: sgc.dequantize_q8(sgc.Quantized(c.q, c.scale.double(), 32)),
              lambda: sgc.rms_norm_backward_q8(x, short, None, v),
              lambda: sgc.rms_norm_backward_q8(x, c, None, v, y=x[:2]),
              lambda: sgc.layer_norm_backward_q8(x, c, w, w, v[:2], v),
              lambda: sgc.layer_norm_backward_q8(x, c, w, w, v, v, dweight=w, accumulate=True),
              lambda: sgc.int8_linear(k, short), lambda: sgc.int8_linear(k, k, w),
              lambda: sgc.int8_linear(k, k, dtype=torch.int32), lambda: sgc.int8_linear(k, k, out=x),
              lambda: sgc.int8_linear(sgc.Quantized(k.q.t(), k.scale), k),
              lambda: sgc.int8_linear(sgc.Quantized(k.q, k.scale[:, 0]), k)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sgc.SGCError):
        sgc.rms_norm(x, out=x, sum_out=x)  # the same buffer for both
    with pytest.raises(sgc.SGCError):
        sgc.rms_norm_backward_q8(x, c, None, v, dx=(t := x.clone()), y=t)


def test_more_rows_than_a_grid_line():
    rows, cols = (1 << 20) + 5, 9
    announce(f"{rows} rows of {cols}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(generator=g)
    pick = torch.tensor([0, 7, (1 << 20) - 1, 1 << 20, rows - 1])
    s = x[pick].cpu()
    q = sgc.rms_norm_q8(x)
    equal_bits(q.q8.q[pick], lm8_ref.rms_q8(s, None, 1e-6)[0], "q")
    for group in (0, 32):
        c = sgc.quantize_q8(x, group=group)
        want, scale = lm8_ref.quantize(s, group)
        equal_bits(c.q[pick], want, "8 bits")
        equal_bits(sgc.dequantize_q8(c, BF16)[pick], lm8_ref.values(want, scale, group).to(BF16), "values")
    w = sgc.quantize_q8(torch.randn(20, cols, generator=gen(1)).cuda(), group=0)
    y = sgc.int8_linear(c if c.group == 0 else sgc.quantize_q8(x, group=0), w, dtype=F32)
    c = sgc.quantize_q8(x[pick.cuda()], group=0)
    ref, tol = lm8_ref.product(c.q, c.scale, w.q, w.scale, None)
    close(y[pick], ref, tol, "product")


@DTYPES
def test_the_longest_rows(dtype):
    """2^20 columns: the norm, 8 bits in groups and a scale a row, and the backward passes from them."""
    rows, cols = 2, 1 << 20
    announce(f"the longest rows {dtype}")
    g = gen(6)
    x, dy = [torch.randn(rows, cols, generator=g).to(dtype) for _ in range(2)]
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    r = sgc.rms_norm(xd, wd)
    (y, rstd), (ty, tr) = lm8_ref.rms(x, w, 1e-6)
    close(r.y, y, ty, "y", dtype)
    close(r.rstd, rstd, tr, "rstd")
    equal_bits(sgc.rms_norm_q8(xd, wd).q8.q, lm8_ref.rms_q8(x, w, 1e-6)[0], "q")
    d = sgc.rms_norm_backward(dyd, xd, wd, r.rstd)
    (dx, dw, _), (tdx, tdw, _) = lm8_ref.backward(dy, x, w, None, r.rstd, None)
    close(d.dx, dx, tdx, "dx", dtype)
    close(d.dweight, dw, tdw, "dweight")
    for group in (0, 32, 256):
        c = sgc.quantize_q8(xd, group=group)
        q, scale = lm8_ref.quantize(x, group)
        equal_bits(c.q, q, "q")
        equal_bits(c.scale, scale, "scale")
        v = lm8_ref.values(q, scale, group)
        equal_bits(sgc.dequantize_q8(c, dtype), v.to(dtype), "values")
        mean, rstd = stats_of(v, "layer")
        k = sgc.layer_norm_backward_q8(dyd, c, wd, b.cuda(), mean.cuda(), rstd.cuda(), want_y=True)
        (dx, dw, db), (tdx, tdw, tdb) = lm8_ref.backward(dy, v, w, mean, rstd, None)
        # the two means over a row are sums of depth(cols) additions
        h = (dbl(v) - dbl(mean)[:, None]) * dbl(rstd)[:, None]
        p = (dbl(dy) * dbl(w)).abs()
        tdx = tdx + lm8_ref.depth(cols) * lm_ref.U * dbl(rstd)[:, None] * (
            p.mean(1, keepdim=True) + h.abs() * (p * h.abs()).mean(1, keepdim=True))
        close(k.dx, dx, tdx, "dx from 8 bits", dtype)
        close(k.dweight, dw, tdw, "dweight from 8 bits")
        close(k.dbias, db, tdb, "dbias from 8 bits")
        y, ty = lm8_ref.normed(v, w, b, mean, rstd)
        close(k.y, y, ty, "y from 8 bits", dtype)
    with pytest.raises(sgc.SGCError):
        sgc.rms_norm(torch.empty(1, cols + 1, dtype=dtype, device="cuda"))
