"""The 64-bit form of distillation with the tail that is right for any distance
of the list from the rest: against the other 64-bit form where both hold, and
its gradient against differences where only this one does."""
import pytest
import torch

import lm_ref
import lm_tail_ref
from test_gpu_lm_tail import far_rows


@pytest.mark.parametrize("gap", [0.0, 5.0, 40.0, 200.0, 600.0])
def test_forms_agree(gap):
    z, idx, val = far_rows([gap] * 3, 50, 5, 0.8, torch.float32, 1)
    g = torch.tensor([1.0, 0.5, 0.0])
    loss, d, tl, td = lm_tail_ref.distill(z, idx, val, 0.8, g)
    loss2, d2, _, _ = lm_ref.distill(z, idx, val, True, 0.8, g=g)
    assert torch.allclose(loss, loss2, rtol=1e-12, atol=1e-12)
    assert torch.allclose(d, d2, rtol=1e-10, atol=1e-14)
    # no tolerance lets a missing tail pass
    u = 1.0 - val.double().exp().sum(1)
    assert (u > 0.01).all() and (tl < 1e-2 * u * (1 + gap)).all()
    assert (td[:2].amax(1) < 1e-2 * u[:2]).all()


@pytest.mark.parametrize("gap", [0.0, 30.0, 90.0, 400.0])
@pytest.mark.parametrize("scale", [0.25, 1.0, 4.0])
def test_gradient_against_differences(gap, scale):
    z, idx, val = far_rows([gap, gap], 11, 3, scale, torch.float64, 2)
    g = torch.tensor([1.0, 0.7], dtype=torch.float64)
    d = lm_tail_ref.distill(z, idx, val, scale, g)[1]
    step = 1e-4 / scale
    for i in range(z.numel()):
        hi, lo = z.clone(), z.clone()
        hi.view(-1)[i] += step
        lo.view(-1)[i] -= step
        want = sum(s * float((lm_tail_ref.distill(x, idx, val, scale, g)[0] * g).sum()) for s, x in ((1, hi), (-1, lo)))
        # differences: (1e-4)^2 third derivatives; 64-bit rounding of a loss below 1e3 over the step
        assert abs(float(d.view(-1)[i]) - want / (2 * step)) < scale * (1e-8 + 1e3 * 2.0 ** -53 / 1e-4 * 4), i
