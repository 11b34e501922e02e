"""More language-model operators of this repository as measured work: their
plain forms, the calls a user makes of the kernels, and the cases.

Three that meet in 8 bits, between a model's body and its loss:

* ``rms``     RMS norm of a residual stream with the addition before it, its
              output in the stream's type or in 8 bits with a scale a row, and
              its gradients;
* ``ckpt``    activations kept in 8 bits with a scale a group of elements (or a
              row), read back, and a norm's backward pass from them, which also
              gives the normed activations again;
* ``linear``  products of 8-bit integers with a scale for each token and each
              channel, alone and after the norm that makes their rows.

``run`` computes them in elementary torch operations in fp32, or, where
``own`` is true, by the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
# the largest listed cases: what a drawn case may cost at most
MOST_NORM = 16384 * 4096
MOST_WEIGHTS = 50000 * 8192
MOST_PRODUCT = 4096 * 4096 * 50000


def listed():
    return [
        # one decoding step of 8 sequences at the width of the recurrent layers
        dict(name="rms_decode", op="rms", pas="forward", rows=8, cols=1024, dtype="bf16", wdtype="fp32",
             residual=True),
        # a training batch of 16384 tokens, forward
        dict(name="rms_train", op="rms", pas="forward", rows=16384, cols=4096, dtype="bf16", wdtype="fp32",
             residual=True),
        # the same batch backward, the residual stream's gradient joined and the weight's summed
        dict(name="rms_train_backward", op="rms", pas="backward", rows=16384, cols=4096, dtype="bf16",
             wdtype="fp32", residual=True),
        # scoring an odd number of tokens: rows in 8 bits for a product
        dict(name="rms_q8", op="rms", pas="q8", rows=10007, cols=1024, dtype="fp16", wdtype="fp16", residual=True),
        # a training batch's activations kept in 8 bits and read back
        dict(name="ckpt_train", op="ckpt", pas="save", rows=16384, cols=4096, dtype="bf16", group=128),
        # that batch's backward pass from the 8 bits, the normed activations given again
        dict(name="ckpt_train_backward", op="ckpt", pas="backward", kind="rms", rows=16384, cols=4096, dtype="bf16",
             wdtype="fp32", group=128, residual=True),
        # the word model's hidden width (650), an odd number of tokens, layer norm, all in fp32
        dict(name="ckpt_word_backward", op="ckpt", pas="backward", kind="layer", rows=20001, cols=650, dtype="fp32",
             wdtype="fp32", group=64, residual=False),
        # the translation model's output weights put into 8 bits, a scale for each channel
        dict(name="ckpt_weights", op="ckpt", pas="save", rows=50000, cols=1024, dtype="fp32", group=0),
        # serving one token: the translation model's head
        dict(name="linear_token", op="linear", pas="product", rows=1, width=1024, out=50000, dtype="bf16",
             bias=False),
        # serving 32 sequences: the norm in 8 bits and the product after it
        dict(name="linear_step", op="linear", pas="step", rows=32, width=4096, out=4096, dtype="fp16", bias=True),
        # the word model's head: a width that is no multiple of 16, logits in fp32
        dict(name="linear_word", op="linear", pas="product", rows=1500, width=650, out=10000, dtype="fp32",
             bias=True),
        # a teacher scores a batch: the largest head
        dict(name="linear_score", op="linear", pas="product", rows=4096, width=4096, out=50000, dtype="bf16",
             bias=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms", "ckpt", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "linear":
        width = _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        out = _log_int(rng, 64, min(131072, MOST_WEIGHTS // width))
        if rng.random() < 0.5:
            out = max(64, out // 8 * 8)
        rows = _log_int(rng, 1, max(1, min(8192, MOST_PRODUCT // (2 * width * out))))
        return dict(op=op, pas=rng.choice(["product", "product", "step"]), rows=rows, width=width, out=out,
                    dtype=dtype, bias=rng.random() < 0.5)
    cols = _log_int(rng, 64, 16384)
    if rng.random() < 0.5:
        cols = max(64, cols // 64 * 64)
    rows = _log_int(rng, 1, max(1, min(32768, MOST_NORM // (2 * cols))))
    wdtype = rng.choice(["fp32", dtype])
    residual = rng.random() < 0.6
    if op == "rms":
        return dict(op=op, pas=rng.choice(["forward", "q8", "backward"]), rows=rows, cols=cols, dtype=dtype,
                    wdtype=wdtype, residual=residual)
    if rng.random() < 0.5:
        return dict(op=op, pas="save", rows=rows, cols=cols, dtype=dtype, group=rng.choice([0, 32, 64, 128, 256]))
    return dict(op=op, pas="backward", kind=rng.choice(["rms", "layer"]), rows=rows, cols=cols, dtype=dtype,
                wdtype=wdtype, group=rng.choice([32, 64, 128, 256]), residual=residual)


# ------------------------------------------------------------------ inputs
def _to_8_bits(x, group):
    """x [rows, cols] as whole numbers up to 127 and a scale a group (0: a row): every operation rounded to fp32."""
    rows, cols = x.shape
    width = group if group else cols
    groups = -(-cols // width)
    p = torch.nn.functional.pad(x.float(), (0, groups * width - cols)).view(rows, groups, width)
    top = p.abs().amax(2, keepdim=True)
    q = torch.round(p * (torch.full_like(top, 127.0) / top))
    q = torch.where(top > 0, q, 0.0).view(rows, groups * width)[:, :cols].to(torch.int8)
    return q, (top / torch.full_like(top, 127.0))[:, :, 0]


def _from_8_bits(q, scale, group):
    if group:
        scale = scale.repeat_interleave(group, dim=1)[:, :q.shape[1]]
    return q.to(scale.dtype) * scale


def _rows_of_8_bits(q):
    """The same rows, each beginning at a multiple of 16 bytes, as a program lays out what a product reads."""
    rows, cols = q.shape
    to = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.int8, device=q.device)
    to[:, :cols] = q
    return to[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    s = dict(case=dict(case))
    rows = case["rows"]

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)

    def stream(cols, dt):
        # a residual stream: some channels far above the others
        loud = torch.where(torch.rand(cols, device="cuda", generator=g) < 0.01, 8.0, 1.0)
        return normal(rows, cols).mul_(loud).to(dt)

    if case["op"] == "linear":
        width, out, dt = case["width"], case["out"], DTYPES[case["dtype"]]
        q, s["wscale"] = _to_8_bits(normal(out, width, std=width ** -0.5), 0)
        s["wq"] = _rows_of_8_bits(q)
        s["bias"] = normal(out, std=0.1) if case["bias"] else None
        if case["pas"] == "step":
            s["x"], s["weight"] = stream(width, dt), normal(width, dtype=dt, mean=1.0, std=0.1)
            s["residual"] = normal(rows, width, dtype=dt)
        else:
            q, s["xscale"] = _to_8_bits(stream(width, torch.float32), 0)
            s["xq"] = _rows_of_8_bits(q)
        return s
    cols, dt = case["cols"], DTYPES[case["dtype"]]
    s["x"] = stream(cols, dt)
    if case["pas"] == "save":
        return s
    s["weight"] = normal(cols, dtype=DTYPES[case["wdtype"]], mean=1.0, std=0.1)
    s["residual"] = s["dsum"] = None
    if case["pas"] != "backward":
        if case["residual"]:
            s["residual"] = normal(rows, cols, dtype=dt)
        return s
    # the forward pass left these
    x = s["x"]
    if case["op"] == "ckpt":
        s["q"], s["scale"] = _to_8_bits(x, case["group"])
        del s["x"]
        if case["kind"] == "layer":
            s["bias"] = normal(cols, dtype=DTYPES[case["wdtype"]], std=0.1)
            s["mean"] = x.double().mean(1).float()
            s["rstd"] = (x.double().var(1, unbiased=False) + EPS).rsqrt().float()
    if case["op"] == "rms" or case["kind"] == "rms":
        s["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
    s["dy"] = normal(rows, cols, dtype=dt)
    if case["residual"]:
        s["dsum"] = normal(rows, cols, dtype=dt)
    return s


# ------------------------------------------------------------- plain forms
def _plain_sum(s):
    x = s["x"]
    return x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)


def _plain_rstd(t):
    return torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)


def _plain_rms(s):
    total = _plain_sum(s)
    t = total.float()
    rstd = _plain_rstd(t)
    y = t * rstd * s["weight"].float()
    return dict(sum=total, y=y.to(total.dtype), rstd=rstd[:, 0])


def _plain_rms_q8(s):
    total = _plain_sum(s)
    t = total.float()
    rstd = _plain_rstd(t)
    q, scale = _to_8_bits(t * s["weight"].float(), 0)
    return total, q, scale * rstd, rstd[:, 0]


def _plain_backward(s, t):
    """Gradients of an RMS norm, or where there is a mean of a layer norm, of t (fp32)."""
    dt = s["dy"].dtype
    dy, rstd, w = s["dy"].float(), s["rstd"][:, None], s["weight"].float()
    layer = s["case"].get("kind") == "layer"
    h = (t - s["mean"][:, None]) * rstd if layer else t * rstd
    v = dy * w
    d = v - h * (v * h).mean(1, keepdim=True)
    if layer:
        d = d - v.mean(1, keepdim=True)
    dx = rstd * d
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    out = dict(dx=dx.to(dt), dweight=(dy * h).sum(0))
    if layer:
        out["dbias"] = dy.sum(0)
    if s["case"]["op"] == "ckpt":
        out["y"] = (h * w + s["bias"].float() if layer else h * w).to(dt)
    return out


def _plain_product(s, xq, xscale, dt):
    y = xq.float() @ s["wq"].float().t()
    y = y * (xscale * s["wscale"].t())
    return (y if s["bias"] is None else y + s["bias"]).to(dt)


def _plain(s):
    case = s["case"]
    if case["op"] == "rms":
        if case["pas"] == "forward":
            return _plain_rms(s)
        if case["pas"] == "backward":
            return _plain_backward(s, s["x"].float())
        total, q, scale, rstd = _plain_rms_q8(s)
        return dict(sum=total, values=_from_8_bits(q, scale, 0).to(total.dtype), scale=scale, rstd=rstd)
    if case["op"] == "ckpt":
        if case["pas"] == "backward":
            return _plain_backward(s, _from_8_bits(s["q"], s["scale"], case["group"]))
        q, scale = _to_8_bits(s["x"], case["group"])
        return dict(values=_from_8_bits(q, scale, case["group"]).to(s["x"].dtype), scale=scale)
    dt = DTYPES[case["dtype"]]
    if case["pas"] == "product":
        return dict(y=_plain_product(s, s["xq"], s["xscale"], dt))
    total, q, scale, _ = _plain_rms_q8(s)
    return dict(sum=total, y=_plain_product(s, q, scale, dt))


# ---------------------------------------------------------- the kernels' calls
def _own(s):
    import compressed_sgd_amd as sgc

    case = s["case"]
    if case["op"] == "rms":
        if case["pas"] == "forward":
            r = sgc.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return dict(sum=r.sum, y=r.y, rstd=r.rstd)
        if case["pas"] == "backward":
            r = sgc.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dsum=s["dsum"])
            return dict(dx=r.dx, dweight=r.dweight)
        r = sgc.rms_norm_q8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        return dict(sum=r.sum, values=sgc.dequantize_q8(r.q8, s["x"].dtype), scale=r.q8.scale, rstd=r.rstd)
    if case["op"] == "ckpt":
        if case["pas"] == "save":
            c = sgc.quantize_q8(s["x"], group=case["group"])
            return dict(values=sgc.dequantize_q8(c, s["x"].dtype), scale=c.scale)
        c = sgc.Quantized(s["q"], s["scale"], case["group"])
        if case["kind"] == "rms":
            r = sgc.rms_norm_backward_q8(s["dy"], c, s["weight"], s["rstd"], dsum=s["dsum"], want_y=True)
            return dict(dx=r.dx, dweight=r.dweight, y=r.y)
        r = sgc.layer_norm_backward_q8(s["dy"], c, s["weight"], s["bias"], s["mean"], s["rstd"], dsum=s["dsum"],
                                       want_y=True)
        return dict(dx=r.dx, dweight=r.dweight, dbias=r.dbias, y=r.y)
    dt, w = DTYPES[case["dtype"]], sgc.Quantized(s["wq"], s["wscale"])
    if case["pas"] == "product":
        return dict(y=sgc.int8_linear(sgc.Quantized(s["xq"], s["xscale"]), w, s["bias"], dtype=dt))
    r = sgc.rms_norm_q8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    return dict(sum=r.sum, y=sgc.int8_linear(r.q8, w, s["bias"], dtype=dt))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    size = DTYPES[case["dtype"]].itemsize
    rows = case["rows"]
    if case["op"] == "linear":
        width, out = case["width"], case["out"]
        product = dict(bytes=out * width + rows * out * size + 4 * out, flops=2 * rows * width * out)
        if case["pas"] == "product":
            product["bytes"] += rows * width + 4 * rows
        else:  # the stream and what is added to it read, the sum written
            product["bytes"] += 3 * rows * width * size + width * size
        return product
    n, cols = rows * case["cols"], case["cols"]
    if case["op"] == "ckpt" and case["pas"] == "save":
        # read, the 8 bits written and read, the values written
        groups = -(-cols // case["group"]) if case["group"] else 1
        return dict(bytes=2 * n * size + 2 * n + 8 * rows * groups, flops=5 * n)
    wsize = DTYPES[case["wdtype"]].itemsize
    if case["op"] == "ckpt":
        groups = -(-cols // case["group"])
        layer = case["kind"] == "layer"
        return dict(bytes=(4 if case["residual"] else 3) * n * size + n + 4 * rows * groups + cols * (wsize + 4)
                    * (2 if layer else 1) + 4 * rows * (2 if layer else 1), flops=(18 if layer else 14) * n)
    if case["pas"] == "forward":
        return dict(bytes=(4 if case["residual"] else 2) * n * size + cols * wsize + 4 * rows, flops=5 * n)
    if case["pas"] == "q8":  # and the values that the 8 bits stand for
        return dict(bytes=(4 if case["residual"] else 2) * n * size + 2 * n + cols * wsize + 12 * rows, flops=8 * n)
    return dict(bytes=(4 if case["residual"] else 3) * n * size + cols * (wsize + 4) + 4 * rows, flops=11 * n)


# ------------------------------------------------------------------ 64 bits
def _exact_8_bits(p, group):
    """The whole numbers and the 64-bit scales of p (fp32).  The definition rounds the factor and the product
    with it to fp32 before the whole number is taken; both are so here too."""
    cols = p.shape[1]
    parts, scales = [], []
    for a in range(0, cols, group or cols):
        part = p[:, a:a + (group or cols)]
        top = part.abs().max(dim=1, keepdim=True).values.double()
        factor = torch.where(top > 0, 127.0 / top, 0.0).float().double()
        parts.append((part.double() * factor).float().double().round())
        scales.append(top / 127.0)
    return torch.cat(parts, 1), torch.cat(scales, 1)


def _exact_values(q, scale, group):
    cols = q.shape[1]
    return torch.cat([q[:, a:a + (group or cols)].double() * scale[:, k:k + 1]
                      for k, a in enumerate(range(0, cols, group or cols))], 1)


def _exact_sum(s):
    x = s["x"].double()
    return x if s["residual"] is None else (x + s["residual"].double())


def _exact_norm_q8(s):
    t = _exact_sum(s).to(s["x"].dtype)
    rstd = 1.0 / torch.sqrt((t.double() ** 2).mean(1, keepdim=True) + EPS)
    q, scale = _exact_8_bits((t.double() * s["weight"].double()).float(), 0)
    return t, q, scale * rstd, rstd[:, 0]


def _exact_product(s, q, scale):
    y = torch.mm(q.double(), s["wq"].double().t())
    y *= scale
    y *= s["wscale"].double()[:, 0]
    return y if s["bias"] is None else y.add_(s["bias"].double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        if case["pas"] == "product":
            return dict(y=_exact_product(s, s["xq"], s["xscale"].double()))
        _, q, scale, _ = _exact_norm_q8(s)
        return dict(sum=_exact_sum(s), y=_exact_product(s, q, scale))
    if case["pas"] == "save":
        q, scale = _exact_8_bits(s["x"].float(), case["group"])
        return dict(values=_exact_values(q, scale, case["group"]), scale=scale)
    if case["pas"] == "q8":
        _, q, scale, rstd = _exact_norm_q8(s)
        return dict(sum=_exact_sum(s), values=q * scale, scale=scale, rstd=rstd)
    w = s["weight"].double()
    if case["pas"] == "forward":
        t = _exact_sum(s).to(s["x"].dtype).double()  # the norm is of the stream as it is kept
        rstd = 1.0 / torch.sqrt((t ** 2).mean(1) + EPS)
        return dict(sum=_exact_sum(s), y=t * w * rstd[:, None], rstd=rstd)
    ckpt = case["op"] == "ckpt"
    t = _exact_values(s["q"], s["scale"].double(), case["group"]) if ckpt else s["x"].double()
    layer = ckpt and case["kind"] == "layer"
    if layer:
        t = t - s["mean"].double()[:, None]
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    h, v = t * rstd, dy * w
    shared = torch.einsum("rc,rc->r", v, h)[:, None] / t.shape[1]
    dx = torch.addcmul(v, h, shared, value=-1.0)
    if layer:
        dx -= v.mean(1, keepdim=True)
    dx *= rstd
    if s["dsum"] is not None:
        dx += s["dsum"].double()
    out = dict(dx=dx, dweight=torch.einsum("rc,rc->c", dy, h))
    if layer:
        out["dbias"] = dy.sum(0)
    if ckpt:
        out["y"] = torch.addcmul(s["bias"].double(), h, w) if layer else h * w
    return out
