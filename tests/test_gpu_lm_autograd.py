"""The language-model operators beside autograd: parameters under no_grad, and
inside an autograd.Function."""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm_ref
from gpu_util import announce

pytestmark = pytest.mark.gpu


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        r = sgc.layer_norm(x, w, b)
        ctx.save_for_backward(x, w, r.mean, r.rstd)
        return r.y

    @staticmethod
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        g = sgc.layer_norm_backward(dy.contiguous(), x, w, mean, rstd)
        return g.dx, g.dweight, g.dbias


def test_norm_inside_a_function():
    announce("layer norm inside an autograd function")
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(33, 130, generator=g), torch.randn(33, 130, generator=g)
    w, b = torch.randn(130, generator=g), torch.randn(130, generator=g)
    leaves = [t.cuda().requires_grad_() for t in (x, w, b)]
    with pytest.raises(ValueError, match="no graph"):
        sgc.layer_norm(*leaves)
    Norm.apply(*leaves).backward(dy.cuda())
    with torch.no_grad():
        r = sgc.layer_norm(*leaves)
    grads, tols = lm_ref.norm_backward(dy, x, w, r.mean, r.rstd)
    for leaf, ref, tol, what in zip(leaves, grads, tols, ("x", "weight", "bias")):
        lm_ref.close(leaf.grad, ref, tol, what)


def in_place_calls():
    x = torch.zeros(6, 40, device="cuda")
    v = torch.ones(6, device="cuda")
    i = torch.arange(12, device="cuda", dtype=torch.int32).view(6, 2)
    tok = torch.zeros(6, dtype=torch.int64, device="cuda")
    st = sgc.token_logprobs(x).stats
    s4 = sgc.distill(x, i, x[:, :2].contiguous()).stats
    out = sgc.token_logprobs(x, tok, top=2)
    return {
        "layer_norm": lambda t: sgc.layer_norm(t, out=t),
        "layer_norm_backward": lambda t: sgc.layer_norm_backward(x, t, None, v, v, dx=t),
        "dweight": lambda t: sgc.layer_norm_backward(x, x, None, v, v, dweight=t.view(-1)[:40], accumulate=True,
                                                     dbias=torch.zeros(40, device="cuda")),
        "token_logprobs_backward": lambda t: sgc.token_logprobs_backward(t, tok, st, None, v, dlogits=t),
        "token_logprobs": lambda t: sgc.token_logprobs(x, tok, top=2, out=sgc.TokenLogprobs(
            out.logp, t.view(-1)[:6], out.stats, out.top_idx, out.top_logp)),
        "distill": lambda t: sgc.distill(t, i, x[:, :2].contiguous(), dloss=v, dlogits=t),
        "distill_backward": lambda t: sgc.distill_backward(t, i, x[:, :2].contiguous(), s4, v, dlogits=t),
    }


@pytest.mark.parametrize("name", ["layer_norm", "layer_norm_backward", "dweight", "token_logprobs_backward",
                                  "token_logprobs", "distill", "distill_backward"])
def test_a_write_into_what_autograd_saved_is_noticed(name):
    """exp keeps its result for its gradient; a call that writes there must not pass unseen."""
    announce(f"in place over a saved tensor: {name}")
    call = in_place_calls()[name]
    leaf = torch.zeros(6, 40, device="cuda", requires_grad=True)
    saved = leaf.exp()
    call(saved.detach())
    with pytest.raises(RuntimeError, match="inplace operation"):
        saved.sum().backward()
