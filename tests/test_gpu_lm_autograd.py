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
