"""The 8-bit operators and RMS norm without a GPU: the formulas that the GPU
tests compare with against differences, the whole numbers' definition at its
edges, and every refusal of the C calls and of the binding (stand-in pointers:
validation fails before any GPU work).
"""
import ctypes as C

import pytest
import torch

import compressed_sgd_amd as sgc
import lm8_ref
from compressed_sgd_amd import lm, lm8
from test_lm_cpu import A, BAD_NORM, INF, MIS, NAN, P, differences, norm_opts

M4 = P(4098)  # fit for 16 bits, not for 32


# ---------------------------------------------------------------- formulas
def test_rms_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g)
    x, w, dy, ds = r(3, 7), r(7), r(3, 7), r(3, 7)

    def f(x, w):
        return (lm8_ref.rms(x, w, 1e-3)[0][0] * dy).sum() + (x * ds).sum()

    rstd = lm8_ref.rms(x, w, 1e-3)[0][1]
    dx, dw, db = lm8_ref.backward(dy, x, w, None, rstd, ds)[0]
    assert db is None
    for got, h, t in ((dx, lambda v: f(v, w), x), (dw, lambda v: f(x, v), w)):
        assert torch.allclose(got.reshape(-1), differences(h, t, range(t.numel())), rtol=1e-6, atol=1e-8)


def test_normed_rows_are_the_norms_own():
    import lm_ref
    g = torch.Generator().manual_seed(2)
    x, w, b = (torch.randn(*s, dtype=torch.float64, generator=g) for s in ((4, 9), (9,), (9,)))
    (y, rstd), _ = lm8_ref.rms(x, w, 1e-6)
    assert torch.allclose(lm8_ref.normed(x, w, None, None, rstd)[0], y, rtol=1e-12)
    (y, mean, rstd), _ = lm_ref.norm(x, w, b, 1e-6)
    assert torch.allclose(lm8_ref.normed(x, w, b, mean, rstd)[0], y, rtol=1e-12)


@pytest.mark.parametrize("group", [0, 32, 64])
def test_whole_numbers_stand_for_their_values(group):
    """Off by at most half a step of the group (and fp32's own rounding); the largest is 127."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 150, generator=g) * torch.logspace(-30, 30, 5)[:, None]
    x[2, :64] = 0.0
    q, scale = lm8_ref.quantize(x, group)
    v = lm8_ref.values(q, scale, group)
    width = group or 150
    for k, a in enumerate(range(0, 150, width)):
        part = x[:, a:a + width]
        top = part.abs().amax(1, keepdim=True)
        off = (v[:, a:a + width].double() - part.double()).abs()
        assert bool((off <= top.double() / 254 * (1 + 2.0 ** -15)).all())
        assert torch.equal(q[:, a:a + width].abs().amax(1, keepdim=True) == 127, top > 0)


def test_whole_numbers_at_the_edges():
    x = torch.zeros(6, 32)
    x[1, 3], x[2, 3], x[3, 3] = NAN, INF, -INF
    x[4, :4] = torch.tensor([1e-45, -1e-45, 2.8e-45, 0.0])  # the smallest numbers there are
    x[5, :3] = torch.tensor([3.4e38, -1.7e38, 1.0])
    q, scale = lm8_ref.quantize(x, 32)
    assert q[:4].abs().max() == 0 and scale[0] == 0 and torch.isnan(scale[1:4]).all()
    assert q[4, :4].tolist() == [64, -64, 127, 0]
    assert q[5, :3].tolist() == [127, -64, 0]


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("bad", BAD_NORM, ids=str)
def test_rms_refuses_options(bad):
    lib = sgc.lib()
    o = norm_opts(**bad)
    assert lib.sgc_rms_norm(C.byref(o), A, 8, A, 8, A, A, 8, P(8192), 8, None, 0, None, A, None) == sgc.EINVAL
    assert lib.sgc_rms_norm_backward_workspace(C.byref(o)) == 0
    assert lib.sgc_rms_norm_backward(C.byref(o), A, 8, A, 8, A, A, A, 8, A, 8, A, A, 1 << 30, None) == sgc.EINVAL


def test_rms_refuses_pointers_and_strides():
    lib = sgc.lib()
    B = P(8192)

    def f(o=norm_opts(), x=A, xs=8, r=A, rs=8, w=A, s=A, ss=8, y=B, ys=8, q=None, qs=0, sc=None, rstd=A):
        return lib.sgc_rms_norm(C.byref(o) if o else None, x, xs, r, rs, w, s, ss, y, ys, q, qs, sc, rstd, None)

    assert f(o=None) == sgc.EINVAL
    for kw in (dict(x=None), dict(x=MIS), dict(xs=7), dict(xs=-8), dict(r=MIS), dict(rs=3), dict(w=MIS), dict(s=MIS),
               dict(ss=0), dict(ss=7), dict(y=None), dict(y=MIS), dict(ys=0), dict(ys=-1), dict(y=A), dict(rstd=MIS),
               dict(q=A, qs=8, sc=A), dict(sc=A), dict(y=None, q=A, qs=8), dict(y=None, sc=A),
               dict(y=None, q=A, qs=7, sc=A), dict(y=None, q=A, qs=0, sc=A), dict(y=None, q=A, qs=8, sc=MIS)):
        assert f(**kw) == sgc.EINVAL, kw
    assert f(o=norm_opts(flags=1)) == sgc.EINVAL
    assert f(o=norm_opts(rows=0), x=None) == sgc.OK
    o = norm_opts()
    need = lib.sgc_rms_norm_backward_workspace(C.byref(o))
    assert need > 0

    def g(dy=A, dys=8, s=A, ss=8, w=A, r=A, ds=A, dss=8, dx=A, dxs=8, dw=A, ws=A, n=need):
        return lib.sgc_rms_norm_backward(C.byref(o), dy, dys, s, ss, w, r, ds, dss, dx, dxs, dw, ws, n, None)

    for kw in (dict(dy=None), dict(s=None), dict(r=None), dict(dy=MIS), dict(dx=MIS), dict(w=MIS), dict(dw=MIS),
               dict(r=MIS), dict(ds=MIS), dict(dss=5), dict(dys=3), dict(ss=-1), dict(dxs=0), dict(ws=P(4100))):
        assert g(**kw) == sgc.EINVAL, kw
    assert g(ws=None) == sgc.ENOSPC
    assert g(n=need - 1) == sgc.ENOSPC


BAD_Q8 = [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=(1 << 20) + 1), dict(dtype=3), dict(group=16),
          dict(group=-1), dict(group=512), dict(group=48)]


@pytest.mark.parametrize("bad", BAD_Q8, ids=str)
def test_q8_refuses_options(bad):
    lib = sgc.lib()
    kw = dict(rows=4, cols=64, dtype=0, group=32) | bad
    o = lm8.Q8Opts(*kw.values())
    assert lib.sgc_quantize_q8(C.byref(o), A, 1 << 21, A, 1 << 21, A, None) == sgc.EINVAL
    assert lib.sgc_dequantize_q8(C.byref(o), A, 1 << 21, A, A, 1 << 21, None) == sgc.EINVAL
    n = lm8.NormQ8Opts(kw["rows"], kw["cols"], kw["dtype"], 0, kw["group"], 1, 0, 0)
    assert lib.sgc_norm_backward_q8_workspace(C.byref(n)) == 0


def test_q8_refuses_pointers_and_strides():
    lib = sgc.lib()
    o = lm8.Q8Opts(4, 64, 1, 32)
    f = lambda x=A, xs=64, q=A, qs=64, s=A: lib.sgc_quantize_q8(C.byref(o), x, xs, q, qs, s, None)
    g = lambda x=A, xs=64, q=A, qs=64, s=A: lib.sgc_dequantize_q8(C.byref(o), q, qs, s, x, xs, None)
    for kw in (dict(x=None), dict(x=MIS), dict(xs=63), dict(xs=-64), dict(q=None), dict(qs=63), dict(qs=-64),
               dict(s=None), dict(s=M4)):
        assert f(**kw) == sgc.EINVAL and g(**kw) == sgc.EINVAL, kw
    assert f(qs=0) == sgc.EINVAL and g(xs=0) == sgc.EINVAL
    assert lib.sgc_quantize_q8(None, A, 64, A, 64, A, None) == sgc.EINVAL
    assert lib.sgc_dequantize_q8(None, A, 64, A, A, 64, None) == sgc.EINVAL
    o = lm8.Q8Opts(0, 64, 1, 32)
    assert f(x=None) == sgc.OK and g(q=None) == sgc.OK


def nq_opts(rows=4, cols=64, dtype=1, wdtype=0, group=32, kind=0, flags=0, reserved=0):
    return lm8.NormQ8Opts(rows, cols, dtype, wdtype, group, kind, flags, reserved)


def test_norm_backward_q8_refusals():
    lib = sgc.lib()
    B = P(8192)

    def f(o, dy=A, dys=64, q=A, qs=64, sc=A, w=A, b=A, m=A, r=A, ds=A, dss=64, dx=A, dxs=64, y=B, ys=64, dw=A, db=A,
          ws=A, n=1 << 30):
        return lib.sgc_norm_backward_q8(C.byref(o) if o else None, dy, dys, q, qs, sc, w, b, m, r, ds, dss, dx, dxs,
                                        y, ys, dw, db, ws, n, None)

    assert f(None) == sgc.EINVAL
    for bad in (dict(rows=-1), dict(cols=0), dict(dtype=3), dict(wdtype=2), dict(group=33), dict(kind=2),
                dict(kind=-1), dict(flags=2), dict(reserved=1)):
        assert f(nq_opts(**bad)) == sgc.EINVAL, bad
        assert lib.sgc_norm_backward_q8_workspace(C.byref(nq_opts(**bad))) == 0
    o = nq_opts()
    for kw in (dict(dy=None), dict(dy=MIS), dict(dys=63), dict(q=None), dict(qs=63), dict(sc=None), dict(sc=M4),
               dict(w=M4), dict(b=M4), dict(m=None), dict(m=M4), dict(r=None), dict(r=M4), dict(ds=MIS),
               dict(dss=1), dict(dx=MIS), dict(dxs=0), dict(y=MIS), dict(ys=0), dict(y=A), dict(dw=M4), dict(db=M4),
               dict(ws=P(4104))):
        assert f(o, **kw) == sgc.EINVAL, kw
    need = lib.sgc_norm_backward_q8_workspace(C.byref(o))
    assert need > 0 and f(o, ws=None) == sgc.ENOSPC and f(o, n=need - 1) == sgc.ENOSPC
    rms = nq_opts(kind=1)  # no mean, bias or dbias there
    for kw in (dict(b=None, db=None), dict(m=None, db=None), dict(m=None, b=None)):
        assert f(rms, **kw) == sgc.EINVAL, kw
    assert lib.sgc_norm_backward_q8_workspace(C.byref(rms)) < need


def test_int8_linear_refusals():
    lib = sgc.lib()

    def f(rows=4, width=64, out=8, dtype=1, reserved=0, x=A, xs=64, xc=A, w=A, ws=64, wc=A, b=A, y=A, ys=8):
        o = lm8.Int8Opts(rows, width, out, dtype, reserved)
        return lib.sgc_int8_linear(C.byref(o), x, xs, xc, w, ws, wc, b, y, ys, None)

    assert lib.sgc_int8_linear(None, A, 64, A, A, 64, A, A, A, 8, None) == sgc.EINVAL
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=1 << 17, xs=1 << 17, ws=1 << 17),
               dict(out=0), dict(out=1 << 31, ys=1 << 31), dict(dtype=3), dict(reserved=1), dict(x=None), dict(xs=63),
               dict(xs=-64), dict(xc=None), dict(xc=M4), dict(w=None), dict(ws=63), dict(ws=-1), dict(wc=None),
               dict(wc=M4), dict(b=M4), dict(y=None), dict(y=MIS), dict(ys=7), dict(ys=0)):
        assert f(**kw) == sgc.EINVAL, kw
    assert f(rows=0, x=None, y=None) == sgc.OK


def test_binding_refuses_host_tensors_and_shapes():
    x, v = torch.zeros(4, 64), torch.zeros(4)
    c = sgc.Quantized(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1))
    for f in (lambda: sgc.rms_norm(x), lambda: sgc.rms_norm_q8(x), lambda: sgc.rms_norm_backward(x, x, None, v),
              lambda: sgc.quantize_q8(x), lambda: sgc.dequantize_q8(c), lambda: sgc.int8_linear(c, c),
              lambda: sgc.rms_norm_backward_q8(x, c, None, v),
              lambda: sgc.layer_norm_backward_q8(x, c, None, None, v, v)):
        with pytest.raises(ValueError, match="device"):
            f()
    with pytest.raises(ValueError, match="group"):
        sgc.int8_linear(sgc.Quantized(c.q, c.scale, 32), c)
    with pytest.raises(ValueError, match="mean"):
        sgc.layer_norm_backward_q8(x, c, None, None, None, v)


def grad_calls():
    x, w, v = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1)
    c = sgc.Quantized(q, s)
    z = lambda t: t.clone().requires_grad_()
    return {
        "rms_norm x": lambda: sgc.rms_norm(z(x)), "rms_norm weight": lambda: sgc.rms_norm(x, z(w)),
        "rms_norm residual": lambda: sgc.rms_norm(x, residual=z(x)), "rms_norm out": lambda: sgc.rms_norm(x, out=z(x)),
        "rms_norm sum_out": lambda: sgc.rms_norm(x, sum_out=z(x)),
        "rms_norm_q8 x": lambda: sgc.rms_norm_q8(z(x)), "rms_norm_q8 weight": lambda: sgc.rms_norm_q8(x, z(w)),
        "rms_norm_backward dy": lambda: sgc.rms_norm_backward(z(x), x, None, v),
        "rms_norm_backward dsum": lambda: sgc.rms_norm_backward(x, x, None, v, dsum=z(x)),
        "rms_norm_backward dweight": lambda: sgc.rms_norm_backward(x, x, None, v, dweight=z(w)),
        "quantize_q8": lambda: sgc.quantize_q8(z(x)),
        "dequantize_q8": lambda: sgc.dequantize_q8(sgc.Quantized(q, z(s))),
        "rms_norm_backward_q8": lambda: sgc.rms_norm_backward_q8(z(x), c, None, v),
        "rms_norm_backward_q8 weight": lambda: sgc.rms_norm_backward_q8(x, c, z(w), v),
        "layer_norm_backward_q8 bias": lambda: sgc.layer_norm_backward_q8(x, c, w, z(w), v, v),
        "layer_norm_backward_q8 y": lambda: sgc.layer_norm_backward_q8(x, c, w, w, v, v, y=z(x)),
        "int8_linear bias": lambda: sgc.int8_linear(c, c, z(v)),
        "int8_linear scale": lambda: sgc.int8_linear(c, sgc.Quantized(q, z(s))),
    }


@pytest.mark.parametrize("name", grad_calls())
def test_a_tensor_that_requires_grad_is_refused(name):
    with pytest.raises(ValueError, match="no graph"):
        grad_calls()[name]()
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        grad_calls()[name]()


@pytest.mark.parametrize("name", ["quantize_q8", "quantize_q8 in groups", "rms_norm_q8"])
def test_a_scale_to_be_written_that_requires_grad_is_refused(name):
    x, q = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8)
    row, groups = torch.zeros(4, 1, requires_grad=True), torch.zeros(4, 2, requires_grad=True)
    f = {"quantize_q8": lambda: sgc.quantize_q8(x, group=0, out=sgc.Quantized(q, row)),
         "quantize_q8 in groups": lambda: sgc.quantize_q8(x, group=32, out=sgc.Quantized(q, groups, 32)),
         "rms_norm_q8": lambda: sgc.rms_norm_q8(x, out=sgc.Quantized(q, row))}[name]
    with pytest.raises(ValueError, match="no graph"):
        f()
    with torch.no_grad(), pytest.raises(ValueError, match="device"):
        f()
