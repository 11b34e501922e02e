"""Limits of the language-model operators' options, without a GPU."""
import ctypes as C

import pytest

import compressed_sgd_amd as sgc
from compressed_sgd_amd import lm


@pytest.mark.parametrize("rows", [512, 4096])
@pytest.mark.parametrize("vocab", [(1 << 31) - 1, (1 << 30) + 1])
@pytest.mark.parametrize("dtype", [lm.F32, lm.BF16])
def test_longest_rows_are_split_however_many_there_are(rows, vocab, dtype):
    """A row (of stride 0, say) whose places a workgroup could not hold in 32 bits is
    split, which takes a workspace."""
    o = lm.LogprobOpts(rows, vocab, dtype, lm.TOKEN_I64, 5, 1.0)
    assert sgc.lib().sgc_token_logprobs_workspace(C.byref(o)) > 2 * rows * 5 * 8
    d = lm.DistillOpts(rows, vocab, dtype, 5, lm.DISTILL_TAIL, 1.0, 1.0, 0)
    assert sgc.lib().sgc_distill_workspace(C.byref(d)) > 2 * rows * 8
