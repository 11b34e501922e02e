"""Limits of the language-model operators' options, without a GPU."""
import ctypes as C

import pytest
import torch

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


def test_a_scale_whose_powers_of_two_overflow_is_refused():
    """The exponent's factor scale / ln 2 has to be finite in fp32."""
    A = C.c_void_p(4096)
    lib = sgc.lib()
    for scale, ok in ((2.3e38, True), (2.4e38, False), (3.4e38, False)):
        o = lm.LogprobOpts(4, 100, lm.F32, lm.TOKEN_I64, 5, scale)
        d = lm.DistillOpts(4, 100, lm.F32, 5, lm.DISTILL_RENORM, scale, 1.0, 0)
        assert (lib.sgc_token_logprobs_workspace(C.byref(o)) != 0) == ok
        assert (lib.sgc_distill_workspace(C.byref(d)) != 0) == ok
        if not ok:
            assert lib.sgc_token_logprobs(C.byref(o), A, 100, A, A, A, A, A, A, A, A, 1 << 30, None) == sgc.EINVAL
            assert lib.sgc_token_logprobs_backward(C.byref(o), A, 100, A, A, A, A, A, A, 100, None) == sgc.EINVAL
            assert lib.sgc_distill(C.byref(d), A, 100, A, A, A, A, A, A, 100, A, A, 1 << 30, None) == sgc.EINVAL
            assert lib.sgc_distill_backward(C.byref(d), A, 100, A, A, A, A, A, 100, None) == sgc.EINVAL


def test_a_workspace_elsewhere_is_refused():
    """The kernels would write to a host address, or past a view's elements."""
    dev = torch.device("cuda", 0)
    buf = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="ws must be"):
        lm._scratch(32, buf, dev, "distill", None, "sgc_distill")
    with pytest.raises(ValueError, match="ws must be"):
        lm._scratch(32, buf[::2], buf.device, "distill", None, "sgc_distill")
    assert lm._scratch(32, buf, buf.device, "distill", None, "sgc_distill") is buf


def test_few_long_rows_need_a_workspace():
    """The split path's refusals are provoked at these sizes: it has to be the one they take."""
    o = lm.LogprobOpts(1, 1 << 20, lm.F32, lm.TOKEN_I64, 8, 1.0)
    d = lm.DistillOpts(1, 1 << 20, lm.F32, 8, lm.DISTILL_RENORM, 1.0, 1.0, 0)
    assert sgc.lib().sgc_token_logprobs_workspace(C.byref(o)) > lm.LM_WS_NONE
    assert sgc.lib().sgc_distill_workspace(C.byref(d)) > lm.LM_WS_NONE
