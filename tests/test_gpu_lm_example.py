"""The example's training step: the loss end's operators and the compression
path together teach a student."""
import os
import sys

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("vocab,width", [(98, 512), (257, 130)], ids=str)
def test_student_learns_through_compressed_gradients(vocab, width):
    import distill_lm

    announce(f"example {vocab} x {width}")
    first, last, bits = distill_lm.train(vocab=vocab, width=width, rows=1024, steps=60, log=announce)
    assert 0 <= last < 0.5 * first
    assert 0 < bits < 3.0   # 5% of 32 bits and their positions
