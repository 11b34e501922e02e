"""The language-model operators at the longest rows their options take."""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm_ref
from gpu_util import announce

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
V = (1 << 31) - 1
GUARD = 1024
# all logits but these are -inf: sums of a handful of terms, wherever they lie
PLACES = [0, 1, 63, 200, 400, 808, 1608, 8191, 8192, 1 << 20, (1 << 30) - 1, 1 << 30, (1 << 30) + 64, (1 << 30) + 328,
          (1 << 30) + 808, (1 << 30) + 1608, V - 8193, V - 300, V - 9, V - 8, V - 7, V - 2, V - 1]


def longest_row():
    """A row of V between guards, and the logits at PLACES."""
    buf = torch.full((GUARD + V + GUARD,), -float("inf"), dtype=BF16, device="cuda")
    z = buf[GUARD:GUARD + V][None]
    vals = (torch.randn(len(PLACES), generator=torch.Generator().manual_seed(1)) * 2).to(BF16)
    z[0, torch.tensor(PLACES, device="cuda")] = vals.cuda()
    buf[:GUARD], buf[GUARD + V:] = 100.0, 100.0  # read by mistake they would be the row's maximum
    return buf, z, vals.double()


def check_guards(buf):
    assert (buf[:GUARD] == 100.0).all() and (buf[GUARD + V:] == 100.0).all()


def test_distill_longest_row():
    announce("distill 1x(2^31 - 1) bf16")
    buf, z, vals = longest_row()
    listed = [2, 11, len(PLACES) - 1]
    idx = torch.tensor([[PLACES[k] for k in listed]], dtype=torch.int32)
    val = torch.tensor([[-1.0, -2.0, -1.5]])
    small = vals[None].to(BF16)
    loss, d, tl, td = lm_ref.distill(small, torch.tensor([listed], dtype=torch.int32), val, True, 1.0)
    obuf = torch.full_like(buf, 100.0)
    out = obuf[GUARD:GUARD + V][None]
    kw = dict(mode=sgc.DISTILL_TAIL, dlogits=out)
    at = torch.tensor(PLACES, device="cuda")
    r = sgc.distill(z, idx.cuda(), val.cuda(), **kw)
    lm_ref.close(r.loss, loss, tl, "loss")
    lm_ref.close(out[:, at], d, td, "dlogits", BF16)
    assert int(torch.count_nonzero(out)) == len(PLACES)
    check_guards(obuf)
    obuf.fill_(100.0)
    sgc.distill_backward(z, idx.cuda(), val.cuda(), r.stats, **kw)
    lm_ref.close(out[:, at], d, td, "dlogits of the backward call", BF16)
    check_guards(obuf)
    obuf.fill_(100.0)
    sgc.distill_backward(z, idx.cuda(), val.cuda(), r.stats, torch.zeros(1, device="cuda"), **kw)
    assert int(torch.count_nonzero(out)) == 0
    check_guards(obuf)
    check_guards(buf)


@pytest.mark.parametrize("rows", [1, 512])
def test_logprobs_longest_row(rows):
    """One, and so many (the same, stride 0) that rows are not split to fill the card."""
    announce(f"logprobs {rows}x(2^31 - 1) bf16")
    buf, z, vals = longest_row()
    tok = torch.tensor([PLACES[r % len(PLACES)] for r in range(rows)])
    r = sgc.token_logprobs(z.expand(rows, V), tok.cuda(), top=5)
    small = torch.tensor([k % len(PLACES) for k in range(rows)])
    sm, (logp, H, idx, tlp), (t_logp, t_H, t_tlp) = lm_ref.logprobs(vals[None].expand(rows, -1), small, 1.0, 5)
    lm_ref.close(r.logp, logp, t_logp, "logp")
    lm_ref.close(r.entropy, H, t_H, "entropy")
    assert torch.equal(r.top_idx.cpu().long(), torch.tensor(PLACES)[idx])
    lm_ref.close(r.top_logp, tlp, t_tlp, "top_logp")
    if rows == 1:
        obuf = torch.full_like(buf, 100.0)
        out = obuf[GUARD:GUARD + V][None]
        g = torch.ones(1, device="cuda")
        sgc.token_logprobs_backward(z, tok.cuda(), r.stats, r.entropy, g, g, dlogits=out)
        d, td = lm_ref.logprobs_backward(sm, small, g.cpu(), g.cpu())
        lm_ref.close(out[:, torch.tensor(PLACES, device="cuda")], d, td, "dlogits", BF16)
        assert int(torch.count_nonzero(out)) == len(PLACES)
        check_guards(obuf)


@pytest.mark.parametrize("rows", [3, 300, 520])
@pytest.mark.parametrize("vocab,dtype", [(131072, BF16), (131072, torch.float16), (65536, torch.float32)], ids=str)
def test_longest_held_rows_are_held_however_many_there_are(rows, vocab, dtype):
    """With the gradient the longest rows that registers hold take one launch, which needs no workspace."""
    announce(f"held rows {rows}x{vocab} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    z = torch.empty(rows, vocab, dtype=dtype, device="cuda").normal_(0.0, 2.0, generator=g)
    idx = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))[:rows * 8].view(rows, 8).int()
    val = torch.log_softmax(torch.randn(rows, 16, generator=torch.Generator().manual_seed(2)), 1)[:, :8].contiguous()
    dl = torch.rand(rows, generator=torch.Generator().manual_seed(3)) + 0.5
    ws = torch.full((sgc.distill_workspace_bytes(rows, vocab, 8, dtype=dtype) + 256,), 0x5A, dtype=torch.uint8,
                    device="cuda")
    out = torch.empty_like(z)
    assert out.data_ptr() % 128 == 0
    r = sgc.distill(z, idx.cuda(), val.cuda(), mode=sgc.DISTILL_TAIL, dloss=dl.cuda(), dlogits=out, ws=ws)
    assert (ws == 0x5A).all()
    pick = torch.tensor([0, rows // 2, rows - 1])
    loss, d, tl, td = lm_ref.distill(z[pick].cpu(), idx[pick], val[pick], True, 1.0, g=dl[pick])
    lm_ref.close(r.loss[pick], loss, tl, "loss")
    lm_ref.close(out[pick], d, td, "dlogits", dtype)
