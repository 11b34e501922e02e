"""The language-model operators of this repository as measured work: their
plain forms, the calls a user makes of the kernels, and the cases.

Three operators at the loss end of a language model whose gradients are then
compressed and exchanged:

* ``norm``      layer norm, forward, and backward with the sums over the rows
                that are the gradients of weight and bias (fp32, as they go
                into the flat gradient);
* ``logprobs``  log probabilities of given tokens, with entropy and the top
                alternatives of every row, and their gradient;
* ``distill``   the divergence from a teacher's top entries, loss and gradient.

``run`` computes them in elementary torch operations in fp32, or, where
``own`` is true, by the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
# the largest listed cases: what a drawn case may cost at most (elements)
MOST_NORM = 16384 * 4096
MOST_LOGITS = 4096 * 131072


def listed():
    return [
        # one decoding step of 8 sequences at the width of the recurrent layers
        dict(name="norm_decode", op="norm", pas="forward", rows=8, cols=1024, dtype="bf16", wdtype="fp32"),
        # a training batch of 16384 tokens, forward
        dict(name="norm_train", op="norm", pas="forward", rows=16384, cols=4096, dtype="bf16", wdtype="fp32"),
        # the same batch's backward pass with the weight's and bias' gradients
        dict(name="norm_train_backward", op="norm", pas="backward", rows=16384, cols=4096, dtype="bf16",
             wdtype="fp32"),
        # the word model's hidden width (650), an odd number of tokens, all in fp32
        dict(name="norm_word_backward", op="norm", pas="backward", rows=20001, cols=650, dtype="fp32",
             wdtype="fp32"),
        # a serving step: 4 sequences, the translation model's vocabulary, 20 alternatives
        dict(name="logprobs_decode", op="logprobs", pas="forward", rows=4, vocab=50000, top=20, dtype="bf16",
             scale=1.0, masked=False),
        # the word model's vocabulary in fp32 with a masked part, 5 alternatives
        dict(name="logprobs_word", op="logprobs", pas="forward", rows=1500, vocab=10000, top=5, dtype="fp32",
             scale=1.25, masked=True),
        # scoring a long prompt over a large vocabulary
        dict(name="logprobs_prompt", op="logprobs", pas="forward", rows=4096, vocab=131072, top=8, dtype="bf16",
             scale=1.0, masked=False),
        # a training step on the log probabilities with an entropy term
        dict(name="logprobs_step", op="logprobs", pas="step", rows=2048, vocab=50000, top=0, dtype="bf16",
             scale=1.0, masked=False),
        # the character model (98 symbols): a small step, loss and gradient
        dict(name="distill_char", op="distill", pas="step", rows=64, vocab=98, top=16, dtype="fp32", scale=0.5,
             tail=False),
        # evaluation: the loss alone, odd vocabulary, the tail counted
        dict(name="distill_eval", op="distill", pas="forward", rows=2000, vocab=10001, top=32, dtype="fp16",
             scale=1.0, tail=True),
        # a training step of the translation model's head, the tail counted
        dict(name="distill_step", op="distill", pas="step", rows=4096, vocab=50000, top=64, dtype="bf16",
             scale=0.5, tail=True),
        # a large vocabulary, renormalised over the teacher's entries
        dict(name="distill_large", op="distill", pas="step", rows=4096, vocab=131072, top=128, dtype="bf16",
             scale=1.0, tail=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "logprobs", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        rows = _log_int(rng, 1, max(1, min(32768, MOST_NORM // (2 * cols))))
        return dict(op=op, pas=rng.choice(["forward", "backward"]), rows=rows, cols=cols, dtype=dtype,
                    wdtype=rng.choice(["fp32", dtype]))
    vocab = _log_int(rng, 98, 200000)
    if rng.random() < 0.5:
        vocab = max(98, vocab // 8 * 8)
    rows = _log_int(rng, 1, max(1, min(8192, MOST_LOGITS // (2 * vocab))))
    scale = rng.choice([1.0, 0.5, 0.75, 1.25])
    if op == "logprobs":
        return dict(op=op, pas=rng.choice(["forward", "forward", "backward", "step"]), rows=rows, vocab=vocab,
                    top=rng.choice([0, 1, 5, 20, 64]), dtype=dtype, scale=scale, masked=rng.random() < 0.4)
    return dict(op=op, pas=rng.choice(["forward", "backward", "step"]), rows=rows, vocab=vocab,
                top=rng.choice([1, 8, 16, 50, 64, 96]), dtype=dtype, scale=scale, tail=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _distinct(rows, k, vocab, g):
    """k distinct tokens a row: one in each of k equal parts of the vocabulary."""
    width = vocab // k
    part = (torch.rand(rows, k, device="cuda", generator=g) * width).long().clamp(max=width - 1)
    return torch.arange(k, device="cuda") * width + part


def _logits(case, g):
    """Logits of a trained model: most of the mass on a few tokens of a row."""
    rows, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    z = torch.empty(rows, vocab, dtype=dt, device="cuda").normal_(0.0, 2.0, generator=g)
    few = _distinct(rows, 12, vocab, g)
    up = torch.empty(rows, 12, device="cuda").uniform_(3.0, 12.0, generator=g)
    return z.scatter_(1, few, up.to(dt))


def _row_norms(x, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = (x.var(1, unbiased=False) + eps).rsqrt()
    return mean.float(), rstd.float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    s = dict(case=dict(case))
    rows = case["rows"]

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)

    if case["op"] == "norm":
        cols, dt, wdt = case["cols"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        s["eps"] = 1e-5
        s["x"] = normal(rows, cols, dtype=dt, mean=0.25, std=1.5)
        s["weight"] = normal(cols, dtype=wdt, mean=1.0, std=0.1)
        s["bias"] = normal(cols, dtype=wdt, std=0.1)
        if case["pas"] == "backward":  # the forward pass left these
            s["dy"] = normal(rows, cols, dtype=dt)
            s["mean"], s["rstd"] = _row_norms(s["x"], s["eps"])
        return s
    s["logits"] = z = _logits(case, g)
    vocab = case["vocab"]
    if case["op"] == "logprobs":
        if case["masked"]:  # tokens that may not be chosen here
            z.masked_fill_(torch.rand(rows, vocab, device="cuda", generator=g) < 0.2, float("-inf"))
        tok = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        best = z.float().argmax(1)
        tok = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.5, best, tok)
        # a masked token is not what a program asks for; every 17th row asks for none (padding)
        tok = torch.where(torch.isinf(z.gather(1, tok[:, None])[:, 0]), best, tok)
        tok[16::17] = -1
        s["tokens"] = tok
        if case["pas"] != "forward":
            s["dlogp"] = normal(rows)
            s["dentropy"] = normal(rows, std=0.1)
        if case["pas"] == "backward":  # the forward pass left these
            s["stats"] = torch.empty(rows, 2, device="cuda")
            s["entropy"] = torch.empty(rows, device="cuda")
            for a in range(0, rows, 256):
                x = z[a:a + 256].double()
                m = x.amax(1, keepdim=True)
                y = (x - m) * case["scale"]
                e = y.exp()
                t = e.sum(1)
                s["stats"][a:a + 256, 0] = m[:, 0].float()
                s["stats"][a:a + 256, 1] = t.float()
                s["entropy"][a:a + 256] = (t.log() - (e * y.clamp(min=-1e4)).sum(1) / t).float()
        return s
    # a teacher's top entries: distinct tokens, their log probabilities, best first; the
    # student has learnt some of them
    k = case["top"]
    idx = _distinct(rows, k, vocab, g)
    v = normal(rows, k, std=2.0).sort(1, descending=True).values
    mass = torch.empty(rows, 1, device="cuda").uniform_(0.6, 0.98, generator=g)
    s["t_val"] = torch.log_softmax(v, 1) + mass.log()
    order = torch.rand(rows, k, device="cuda", generator=g).argsort(1)
    idx = idx.gather(1, order)
    s["t_idx"] = idx.to(torch.int32)
    z.scatter_(1, idx, (v + normal(rows, k) + 6.0).to(z.dtype))
    if case["pas"] != "forward":
        s["dloss"] = torch.empty(rows, device="cuda").uniform_(0.5, 1.5, generator=g)
        s["dloss"][16::17] = 0.0  # padding
    if case["pas"] == "backward":  # the forward pass left these: maximum, sum, sum outside the list
        s["stats"] = torch.ones(rows, 4, device="cuda")
        for a in range(0, rows, 256):
            x = z[a:a + 256].double()
            m = x.amax(1, keepdim=True)
            e = ((x - m) * case["scale"]).exp()
            s["stats"][a:a + 256, 0] = m[:, 0].float()
            s["stats"][a:a + 256, 1] = e.sum(1).float()
            s["stats"][a:a + 256, 2] = e.scatter(1, idx[a:a + 256], 0.0).sum(1).float()
    return s


# ------------------------------------------------------------- plain forms
def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return dict(y=y.to(s["x"].dtype), mean=mean[:, 0], rstd=rstd[:, 0])


def _plain_norm_backward(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    w = dy * s["weight"].float()
    dx = rstd * (w - w.mean(1, keepdim=True) - xhat * (w * xhat).mean(1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xhat).sum(0), dbias=dy.sum(0))


def _plain_logprobs(s):
    case, logits, tok = s["case"], s["logits"], s["tokens"]
    z = logits.float()
    m = z.amax(1, keepdim=True)
    y = (z - m) * case["scale"]
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    log = torch.log(total)
    given = y.gather(1, tok.clamp(min=0)[:, None]) - log
    out = dict(logp=torch.where(tok >= 0, given[:, 0], 0.0),
               entropy=log[:, 0] - (e * torch.clamp(y, min=-1e4)).sum(1) / total[:, 0])
    if case["top"]:
        # unique keys: the value's order, then the lower token first
        b = (z + 0.0).view(torch.int32)
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * (1 << 32)
        key += (1 << 31) - torch.arange(z.shape[1], device=z.device)
        best = torch.topk(key, case["top"], dim=1).values
        idx = (1 << 31) - (best & 0xFFFFFFFF)
        out["top_idx"] = idx.int()
        out["top_logp"] = y.gather(1, idx) - log
    return out, m, total


def _plain_logprobs_backward(s, m, total, entropy):
    case, tok = s["case"], s["tokens"]
    y = (s["logits"].float() - m) * case["scale"]
    p = torch.exp(y) / total
    lp = torch.clamp(y, min=-1e4) - torch.log(total)
    g = torch.where(tok >= 0, s["dlogp"], 0.0)[:, None]
    dz = -p * (g + s["dentropy"][:, None] * (lp + entropy[:, None]))
    dz.scatter_add_(1, tok.clamp(min=0)[:, None], g)
    return (dz * case["scale"]).to(s["logits"].dtype)


def _plain_teacher(s):
    v = s["t_val"].float()
    if s["case"]["tail"]:
        t = torch.exp(v)
        return t, v, torch.clamp(1.0 - t.sum(1, keepdim=True), min=0.0)
    t = torch.exp(v - v.amax(1, keepdim=True))
    t = t / t.sum(1, keepdim=True)
    return t, torch.log(t), torch.zeros_like(v[:, :1])


def _plain_distill(s):
    case, idx = s["case"], s["t_idx"].long()
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    y = (z - m) * case["scale"]
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    outside = e.scatter(1, idx, 0.0).sum(1, keepdim=True)
    t, log_t, u = _plain_teacher(s)
    log = torch.log(total)
    loss = (t * (log_t - (y.gather(1, idx) - log))).sum(1)
    rest = u * (torch.log(u) - (torch.log(outside) - log))
    loss = loss + torch.where((u > 0) & (outside > 0), rest, 0.0)[:, 0]
    return loss, m, total, outside


def _plain_distill_backward(s, m, total, outside):
    case, idx = s["case"], s["t_idx"].long()
    t, _, u = _plain_teacher(s)
    e = torch.exp((s["logits"].float() - m) * case["scale"])
    a = (t.sum(1, keepdim=True) + u) / total
    dz = e * (a - torch.where(outside > 0, u / outside, 0.0))
    dz.scatter_(1, idx, e.gather(1, idx) * a - t)
    return (dz * (s["dloss"][:, None] * case["scale"])).to(s["logits"].dtype)


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        return _plain_norm(s) if case["pas"] == "forward" else _plain_norm_backward(s)
    if case["op"] == "logprobs":
        if case["pas"] == "backward":
            m, total = s["stats"][:, :1], s["stats"][:, 1:2]
            return dict(dlogits=_plain_logprobs_backward(s, m, total, s["entropy"]))
        out, m, total = _plain_logprobs(s)
        if case["pas"] == "step":
            out["dlogits"] = _plain_logprobs_backward(s, m, total, out["entropy"])
        return out
    if case["pas"] == "backward":
        st = s["stats"]
        return dict(dlogits=_plain_distill_backward(s, st[:, :1], st[:, 1:2], st[:, 2:3]))
    loss, m, total, outside = _plain_distill(s)
    if case["pas"] == "forward":
        return dict(loss=loss)
    return dict(loss=loss, dlogits=_plain_distill_backward(s, m, total, outside))


# ---------------------------------------------------------- the kernels' calls
def _own(s):
    import compressed_sgd_amd as sgc

    case = s["case"]
    if case["op"] == "norm":
        if case["pas"] == "forward":
            r = sgc.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"])
            return dict(y=r.y, mean=r.mean, rstd=r.rstd)
        r = sgc.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return dict(dx=r.dx, dweight=r.dweight, dbias=r.dbias)
    if case["op"] == "logprobs":
        out, stats, entropy = {}, s.get("stats"), s.get("entropy")
        if case["pas"] != "backward":
            r = sgc.token_logprobs(s["logits"], s["tokens"], scale=case["scale"], top=case["top"])
            out = dict(logp=r.logp, entropy=r.entropy)
            if case["top"]:
                out.update(top_idx=r.top_idx, top_logp=r.top_logp)
            stats, entropy = r.stats, r.entropy
        if case["pas"] != "forward":
            out["dlogits"] = sgc.token_logprobs_backward(s["logits"], s["tokens"], stats, entropy, s["dlogp"],
                                                         s["dentropy"], scale=case["scale"])
        return out
    mode = sgc.DISTILL_TAIL if case["tail"] else sgc.DISTILL_RENORM
    if case["pas"] == "backward":
        return dict(dlogits=sgc.distill_backward(s["logits"], s["t_idx"], s["t_val"], s["stats"], s["dloss"],
                                                 mode=mode, scale=case["scale"]))
    if case["pas"] == "forward":
        return dict(loss=sgc.distill(s["logits"], s["t_idx"], s["t_val"], mode=mode, scale=case["scale"]).loss)
    r = sgc.distill(s["logits"], s["t_idx"], s["t_val"], mode=mode, scale=case["scale"], dloss=s["dloss"])
    return dict(loss=r.loss, dlogits=r.dlogits)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    size = DTYPES[case["dtype"]].itemsize
    rows = case["rows"]
    if case["op"] == "norm":
        cols, wsize = case["cols"], DTYPES[case["wdtype"]].itemsize
        n = rows * cols
        if case["pas"] == "forward":
            return dict(bytes=2 * n * size + 2 * cols * wsize + 8 * rows, flops=8 * n)
        return dict(bytes=3 * n * size + cols * (wsize + 8) + 8 * rows, flops=14 * n)
    n, top = rows * case["vocab"], case["top"]
    if case["op"] == "logprobs":
        one = n * size + rows * 16 + rows * top * 8
        if case["pas"] == "forward":
            return dict(bytes=one, flops=6 * n)
        # a step reads the logits once and writes their gradient once
        return dict(bytes=2 * n * size + rows * 32, flops=(6 if case["pas"] == "backward" else 12) * n)
    one = n * size + rows * top * 8 + rows * 4
    if case["pas"] == "forward":
        return dict(bytes=one, flops=5 * n)
    return dict(bytes=one + n * size + rows * 4, flops=(5 if case["pas"] == "backward" else 10) * n)


# ------------------------------------------------------------------ 64 bits
def _exact_norm(s, case):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    if case["pas"] == "forward":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = 1.0 / torch.sqrt(var + s["eps"])
        return dict(y=torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w), mean=mean, rstd=rstd)
    dy, rstd = s["dy"].double(), s["rstd"].double()
    h = (x - s["mean"].double()[:, None]) * rstd[:, None]
    wdy = dy * w
    n = x.shape[1]
    c1, c2 = wdy.sum(1) / n, (wdy * h).sum(1) / n
    dx = (wdy - torch.addcmul(c1[:, None], h, c2[:, None])) * rstd[:, None]
    return dict(dx=dx, dweight=torch.einsum("rc,rc->c", dy, h), dbias=dy.sum(0))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    rows, parts = case["rows"], []
    for a in range(0, rows, 256):
        r = slice(a, min(rows, a + 256))
        x = s["logits"][r].double() * case["scale"]
        if case["op"] == "logprobs":
            parts.append(_exact_logprobs(s, case, r, x))
        else:
            parts.append(_exact_distill(s, case, r, x))
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_logprobs(s, case, r, x):
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    tok = s["tokens"][r]
    has = tok >= 0
    h = -torch.where(p > 0, p * lp, 0.0).sum(1)
    out = {}
    if case["pas"] != "backward":
        out["logp"] = torch.where(has, lp[torch.arange(len(tok), device=lp.device), tok.clamp(min=0)], 0.0)
        out["entropy"] = h
        if case["top"]:
            out["top_idx"] = None
            out["top_logp"] = torch.topk(lp, case["top"], dim=1).values
    if case["pas"] != "forward":
        hot = torch.zeros_like(p)
        hot[torch.arange(len(tok), device=lp.device)[has], tok[has]] = 1.0
        gl = torch.where(has, s["dlogp"][r].double(), 0.0)[:, None]
        gh = s["dentropy"][r].double()[:, None]
        inner = torch.where(p > 0, p * (lp + h[:, None]), 0.0)
        out["dlogits"] = case["scale"] * (gl * (hot - p) - gh * inner)
    return out


def _exact_distill(s, case, r, x):
    lq = torch.log_softmax(x, 1)
    idx = s["t_idx"][r].long()
    v = s["t_val"][r].double()
    inside = torch.zeros_like(lq, dtype=torch.bool).scatter_(1, idx, True)
    out_q = torch.where(inside, 0.0, lq.exp()).sum(1)
    if case["tail"]:
        t = v.exp()
        u = (1.0 - t.sum(1)).clamp(min=0.0)
    else:
        v = torch.log_softmax(v, 1)
        t, u = v.exp(), torch.zeros(len(v), dtype=v.dtype, device=v.device)
    out = {}
    tail = (u > 0) & (out_q > 0)
    if case["pas"] != "backward":
        rest = torch.where(tail, u * (u.log() - out_q.log()), 0.0)
        out["loss"] = (t * (v - lq.gather(1, idx))).sum(1) + rest
    if case["pas"] != "forward":
        share = torch.where(tail, u / out_q, 0.0)[:, None]
        q = lq.exp()
        target = torch.where(inside, 0.0, q * share).scatter_(1, idx, t)
        mass = (t.sum(1) + u)[:, None]
        out["dlogits"] = (q * mass - target) * (s["dloss"][r].double()[:, None] * case["scale"])
    return out
