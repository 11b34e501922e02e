"""The language-model operators without a GPU: the 64-bit forms that the GPU
tests compare with are checked against differences, and every refusal of the
C calls and of the binding is provoked (stand-in pointers: validation fails
before any GPU work).
"""
import ctypes as C

import pytest
import torch

import compressed_sgd_amd as sgc
import lm_ref
from compressed_sgd_amd import lm

P = C.c_void_p
A = P(4096)
MIS = P(4097)
NAN, INF = float("nan"), float("inf")


def differences(f, x, at, step=1e-5):
    out = []
    for i in at:
        hi, lo = x.clone(), x.clone()
        hi.view(-1)[i] += step
        lo.view(-1)[i] -= step
        out.append((f(hi) - f(lo)) / (2 * step))
    return torch.stack(out)


def test_norm_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 7, dtype=torch.float64, generator=g)
    w = torch.randn(7, dtype=torch.float64, generator=g)
    b = torch.randn(7, dtype=torch.float64, generator=g)
    dy = torch.randn(3, 7, dtype=torch.float64, generator=g)

    def y(x, w, b):
        return (lm_ref.norm(x, w, b, 1e-3)[0][0] * dy).sum()

    _, mean, rstd = lm_ref.norm(x, w, b, 1e-3)[0]
    dx, dw, db = lm_ref.norm_backward(dy, x, w, mean, rstd)[0]
    for got, f, t in ((dx, lambda v: y(v, w, b), x), (dw, lambda v: y(x, v, b), w), (db, lambda v: y(x, w, v), b)):
        want = differences(f, t, range(t.numel()))
        assert torch.allclose(got.reshape(-1), want, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_logprobs_gradient_formula_against_differences(scale):
    g = torch.Generator().manual_seed(2)
    z = torch.randn(4, 9, dtype=torch.float64, generator=g) * 2
    z[1, 3] = -INF
    tok = torch.tensor([2, 0, -1, 8])
    gl, gh = torch.randn(4, dtype=torch.float64, generator=g), torch.randn(4, dtype=torch.float64, generator=g)

    def f(z):
        _, (logp, H, _, _), _ = lm_ref.logprobs(z, tok, scale, 0)
        return (logp * gl + H * gh).sum()

    d = lm_ref.logprobs_backward(lm_ref.logprobs(z, tok, scale, 0)[0], tok, gl, gh)[0]
    at = [i for i in range(z.numel()) if torch.isfinite(z.view(-1)[i])]
    assert torch.allclose(d.view(-1)[at], differences(f, z, at), rtol=1e-6, atol=1e-8)
    assert d[1, 3] == 0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_distill_gradient_formula_against_differences(tail, scale):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(3, 11, dtype=torch.float64, generator=g) * 2
    idx = torch.tensor([[4, 0, 9], [1, -1, 10], [-1, -1, 5]], dtype=torch.int32)
    val = torch.log_softmax(torch.randn(3, 11, generator=g), 1)[:, :3].contiguous()
    gl = torch.randn(3, dtype=torch.float64, generator=g)

    def f(z):
        return (lm_ref.distill(z, idx, val, tail, scale)[0] * gl).sum()

    d = lm_ref.distill(z, idx, val, tail, scale, g=gl)[1]
    assert torch.allclose(d.view(-1), differences(f, z, range(z.numel())), rtol=1e-6, atol=1e-8)


# ------------------------------------------------------------------ refusals
def norm_opts(rows=4, cols=8, dtype=0, wdtype=0, eps=1e-5, flags=0):
    return lm.NormOpts(rows, cols, dtype, wdtype, eps, flags)


BAD_NORM = [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=(1 << 20) + 1), dict(dtype=3),
            dict(dtype=-1), dict(dtype=1, wdtype=2), dict(wdtype=1), dict(eps=-1e-5), dict(eps=NAN), dict(eps=INF),
            dict(flags=2)]


@pytest.mark.parametrize("bad", BAD_NORM, ids=str)
def test_norm_refuses_options(bad):
    lib = sgc.lib()
    o = norm_opts(**bad)
    assert lib.sgc_layer_norm(C.byref(o), A, 8, A, A, A, 8, A, A, None) == sgc.EINVAL
    assert lib.sgc_layer_norm_backward_workspace(C.byref(o)) == 0
    assert lib.sgc_layer_norm_backward(C.byref(o), A, 8, A, 8, A, A, A, A, 8, A, A, A, 1 << 30, None) == sgc.EINVAL


def test_norm_refuses_pointers_and_strides():
    lib = sgc.lib()
    o = norm_opts()
    f = lambda o=o, x=A, xs=8, w=A, b=A, y=A, ys=8, m=A, r=A: \
        lib.sgc_layer_norm(C.byref(o) if o else None, x, xs, w, b, y, ys, m, r, None)
    assert f(o=None) == sgc.EINVAL
    for kw in (dict(x=None), dict(y=None), dict(x=MIS), dict(y=MIS), dict(w=MIS), dict(b=MIS), dict(m=MIS),
               dict(r=MIS), dict(xs=7), dict(xs=-8), dict(ys=7), dict(ys=0), dict(ys=-8)):
        assert f(**kw) == sgc.EINVAL, kw
    assert f(o=norm_opts(flags=1)) == sgc.EINVAL            # nothing is added in the forward call
    assert f(o=norm_opts(rows=0), x=None, y=None) == sgc.OK
    need = lib.sgc_layer_norm_backward_workspace(C.byref(o))
    assert need > 0
    g = lambda dy=A, dys=8, x=A, xs=8, w=A, m=A, r=A, dx=A, dxs=8, dw=A, db=A, ws=A, n=need: \
        lib.sgc_layer_norm_backward(C.byref(o), dy, dys, x, xs, w, m, r, dx, dxs, dw, db, ws, n, None)
    for kw in (dict(dy=None), dict(x=None), dict(m=None), dict(r=None), dict(dy=MIS), dict(dx=MIS), dict(w=MIS),
               dict(dw=MIS), dict(db=MIS), dict(m=MIS), dict(r=MIS), dict(dys=3), dict(xs=-1), dict(dxs=0),
               dict(ws=P(4100))):
        assert g(**kw) == sgc.EINVAL, kw
    assert g(ws=None) == sgc.ENOSPC
    assert g(n=need - 1) == sgc.ENOSPC


def lp_opts(rows=4, vocab=100, dtype=0, token_type=1, top=5, scale=1.0):
    return lm.LogprobOpts(rows, vocab, dtype, token_type, top, scale)


BAD_LP = [dict(rows=-1), dict(rows=1 << 31), dict(vocab=0, top=0), dict(vocab=1 << 31), dict(dtype=3),
          dict(token_type=2), dict(top=-1), dict(top=101), dict(vocab=1000, top=257), dict(scale=0.0),
          dict(scale=-1.0), dict(scale=NAN), dict(scale=INF)]


@pytest.mark.parametrize("bad", BAD_LP, ids=str)
def test_logprobs_refuses_options(bad):
    lib = sgc.lib()
    o = lp_opts(**bad)
    assert lib.sgc_token_logprobs_workspace(C.byref(o)) == 0
    assert lib.sgc_token_logprobs(C.byref(o), A, 1 << 31, A, A, A, A, A, A, A, A, 1 << 30, None) == sgc.EINVAL
    assert lib.sgc_token_logprobs_backward(C.byref(o), A, 1 << 31, A, A, A, A, A, A, 1 << 31, None) == sgc.EINVAL


def test_logprobs_refuses_pointers_and_strides():
    lib = sgc.lib()
    o = lp_opts()
    need = lib.sgc_token_logprobs_workspace(C.byref(o))
    assert need >= 1
    f = lambda o=o, z=A, zs=100, tok=A, lp=A, H=A, st=A, ti=A, tl=A, ds=A, ws=A, n=1 << 30: \
        lib.sgc_token_logprobs(C.byref(o) if o else None, z, zs, tok, lp, H, st, ti, tl, ds, ws, n, None)
    assert f(o=None) == sgc.EINVAL
    for kw in (dict(z=None), dict(z=MIS), dict(zs=99), dict(zs=-100), dict(tok=None), dict(lp=None), dict(tok=P(4100)),
               dict(lp=MIS), dict(H=MIS), dict(st=MIS), dict(ti=None), dict(tl=None), dict(ti=MIS), dict(tl=MIS),
               dict(ds=MIS)):
        assert f(**kw) == sgc.EINVAL, kw
    assert f(o=lp_opts(rows=0), z=None) == sgc.OK
    g = lambda z=A, zs=100, tok=A, st=A, H=A, dl=A, dh=A, dz=A, dzs=100: \
        lib.sgc_token_logprobs_backward(C.byref(o), z, zs, tok, st, H, dl, dh, dz, dzs, None)
    for kw in (dict(z=None), dict(zs=5), dict(tok=None), dict(tok=P(4100)), dict(st=None), dict(H=None), dict(dz=None),
               dict(dzs=0), dict(dzs=99), dict(dz=MIS), dict(dl=MIS), dict(dh=MIS), dict(st=MIS), dict(H=MIS)):
        assert g(**kw) == sgc.EINVAL, kw


def di_opts(rows=4, vocab=100, dtype=0, top=5, mode=0, scale=1.0, teacher_scale=1.0, reserved=0):
    return lm.DistillOpts(rows, vocab, dtype, top, mode, scale, teacher_scale, reserved)


BAD_DI = [dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=1 << 31), dict(dtype=3), dict(top=0),
          dict(top=257), dict(mode=2), dict(mode=-1), dict(scale=0.0), dict(scale=NAN), dict(scale=INF),
          dict(teacher_scale=0.0), dict(teacher_scale=NAN), dict(mode=1, teacher_scale=0.5), dict(reserved=1)]


@pytest.mark.parametrize("bad", BAD_DI, ids=str)
def test_distill_refuses_options(bad):
    lib = sgc.lib()
    o = di_opts(**bad)
    assert lib.sgc_distill_workspace(C.byref(o)) == 0
    assert lib.sgc_distill(C.byref(o), A, 1 << 31, A, A, A, A, A, A, 1 << 31, A, A, 1 << 30, None) == sgc.EINVAL
    assert lib.sgc_distill_backward(C.byref(o), A, 1 << 31, A, A, A, A, A, 1 << 31, None) == sgc.EINVAL


def test_distill_refuses_pointers_and_strides():
    lib = sgc.lib()
    o = di_opts()
    f = lambda o=o, z=A, zs=100, ti=A, tv=A, lo=A, st=A, dl=A, dz=A, dzs=100, ds=A: \
        lib.sgc_distill(C.byref(o) if o else None, z, zs, ti, tv, lo, st, dl, dz, dzs, ds, A, 1 << 30, None)
    assert f(o=None) == sgc.EINVAL
    for kw in (dict(z=None), dict(z=MIS), dict(zs=99), dict(zs=-1), dict(ti=None), dict(tv=None), dict(ti=MIS),
               dict(tv=MIS), dict(lo=None), dict(lo=MIS), dict(st=MIS), dict(dl=MIS), dict(dz=MIS), dict(dzs=0),
               dict(dzs=99), dict(ds=MIS)):
        assert f(**kw) == sgc.EINVAL, kw
    assert f(o=di_opts(rows=0), z=None) == sgc.OK
    g = lambda z=A, zs=100, ti=A, tv=A, st=A, dl=A, dz=A, dzs=100: \
        lib.sgc_distill_backward(C.byref(o), z, zs, ti, tv, st, dl, dz, dzs, None)
    for kw in (dict(z=None), dict(zs=99), dict(ti=None), dict(tv=None), dict(st=None), dict(st=MIS), dict(dl=MIS),
               dict(dz=None), dict(dz=MIS), dict(dzs=0)):
        assert g(**kw) == sgc.EINVAL, kw


def test_workspace_is_enforced_where_one_is_needed():
    """Few long rows are split over workgroups, which meet in a workspace."""
    lib = sgc.lib()
    o = lp_opts(rows=1, vocab=1 << 20, top=8)
    need = lib.sgc_token_logprobs_workspace(C.byref(o))
    if need != sgc.lm.LM_WS_NONE:
        f = lambda ws, n: lib.sgc_token_logprobs(C.byref(o), A, 1 << 20, A, A, A, A, A, A, A, ws, n, None)
        assert f(None, need) == sgc.ENOSPC and f(A, need - 1) == sgc.ENOSPC and f(P(4100), need) == sgc.EINVAL
    d = di_opts(rows=1, vocab=1 << 20, top=8)
    need = lib.sgc_distill_workspace(C.byref(d))
    if need != sgc.lm.LM_WS_NONE:
        f = lambda ws, n: lib.sgc_distill(C.byref(d), A, 1 << 20, A, A, A, A, A, None, 0, A, ws, n, None)
        assert f(None, need) == sgc.ENOSPC and f(A, need - 1) == sgc.ENOSPC and f(P(4100), need) == sgc.EINVAL


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(4, 8)
    v = torch.zeros(4)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: sgc.layer_norm(x), lambda: sgc.layer_norm_backward(x, x, None, v, v),
              lambda: sgc.token_logprobs(x), lambda: sgc.token_logprobs_backward(x, None, x, None, None),
              lambda: sgc.distill(x, i, x), lambda: sgc.distill_backward(x, i, x, x)):
        with pytest.raises(ValueError):
            f()
