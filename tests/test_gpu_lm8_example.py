"""The example in 8 bits runs, and the gradient that it puts together is that of its loss."""
import os
import sys

import pytest
import torch

import lm8_ref
from gpu_util import announce
from lm_ref import U, close, dbl

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_example_in_8_bits_runs():
    import distill_lm

    announce("example in 8 bits")
    first, last, bits = distill_lm.train(vocab=98, width=130, rows=256, steps=3, workers=2, bits=8, log=announce)
    assert first >= 0 and last >= 0 and 0 < bits < 32


def test_gradient_of_the_8_bit_student():
    """Against the formulas in 64 bits, from the values that the 8 bits stand for and the logits' gradient."""
    import distill_lm

    announce("gradient of the 8-bit student")
    vocab, width, rows = 60, 130, 90
    gen = torch.Generator(device="cuda").manual_seed(3)
    student = distill_lm.Student8.make(vocab, width, gen)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    z, (kept, rstd) = student.logits(tokens)
    dlogits = torch.empty_like(z).normal_(0.0, 1.0, generator=gen)
    out = torch.full_like(student.flat, 7.0)
    student.gradient(tokens, (kept, rstd), dlogits, out)

    x = lm8_ref.values(kept.q, kept.scale, 64)
    w = student.part(student.flat, 1).cpu()
    d, head = dbl(dlogits), dbl(student.part(student.flat, 3).bfloat16())
    half = 2.0 ** -8  # a rounding to bfloat16
    dy = d @ head
    t_dy = half * dy.abs() + vocab * U * (d.abs() @ head.abs())
    (dx, dw, _), (t_dx, t_dw, _) = lm8_ref.backward(dy, x, w, None, rstd, None)
    # what dy's error does to them, by the same formulas
    h, rs, aw = (dbl(x) * dbl(rstd)[:, None]).abs(), dbl(rstd)[:, None], dbl(w).abs()
    t_dx = t_dx + rs * (t_dy * aw + h * (t_dy * aw * h).mean(1, keepdim=True))
    t_dx = t_dx + half * (dx.abs() + t_dx)
    close(student.part(out, 1), dw, t_dw + (t_dy * h).sum(0), "the weight's gradient")
    assert not student.part(out, 2).any()
    y, t_y = lm8_ref.normed(x, w, None, None, rstd)
    t_y = t_y + half * (y.abs() + t_y)
    dh = d.t() @ y
    t_dh = d.abs().t() @ t_y + rows * U * (d.abs().t() @ y.abs())
    close(student.part(out, 3), dh, t_dh + half * (dh.abs() + t_dh), "the head's gradient")
    add = lambda t: torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, tokens.cpu(), t)  # noqa: E731
    close(student.part(out, 0), add(dx), add(t_dx) + rows * U * add(dx.abs() + t_dx), "the embedding's gradient")
