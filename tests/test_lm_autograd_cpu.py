"""The language-model operators record no graph: a tensor that requires grad is
refused while grad mode is on, and only then."""
import pytest
import torch

import compressed_sgd_amd as sgc


def calls():
    x, w, v = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    i, s2, s4 = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 4)
    z = lambda t: t.clone().requires_grad_()
    return {
        "layer_norm x": lambda: sgc.layer_norm(z(x)), "layer_norm weight": lambda: sgc.layer_norm(x, z(w)),
        "layer_norm bias": lambda: sgc.layer_norm(x, w, z(w)), "layer_norm out": lambda: sgc.layer_norm(x, out=z(x)),
        "layer_norm_backward dy": lambda: sgc.layer_norm_backward(z(x), x, None, v, v),
        "layer_norm_backward weight": lambda: sgc.layer_norm_backward(x, x, z(w), v, v),
        "layer_norm_backward dweight": lambda: sgc.layer_norm_backward(x, x, w, v, v, dweight=z(w)),
        "token_logprobs": lambda: sgc.token_logprobs(z(x)),
        "token_logprobs_backward": lambda: sgc.token_logprobs_backward(z(x), None, s2, None, None),
        "token_logprobs_backward dlogp": lambda: sgc.token_logprobs_backward(x, None, s2, None, z(v)),
        "distill": lambda: sgc.distill(z(x), i, s2), "distill t_val": lambda: sgc.distill(x, i, z(s2)),
        "distill dloss": lambda: sgc.distill(x, i, s2, dloss=z(v)),
        "distill_backward": lambda: sgc.distill_backward(z(x), i, s2, s4),
        "distill_backward dlogits": lambda: sgc.distill_backward(x, i, s2, s4, dlogits=z(x)),
    }


@pytest.mark.parametrize("name", calls())
def test_a_tensor_that_requires_grad_is_refused(name):
    with pytest.raises(ValueError, match="no graph"):
        calls()[name]()
    with torch.no_grad(), pytest.raises(ValueError, match="device"):  # host tensors: the next refusal
        calls()[name]()
