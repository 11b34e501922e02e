"""Layer norm of fp32 rows around the widths where the shape of a workgroup
changes, rows of whole vectors and not, few and many rows."""
import pytest
import torch

import compressed_sgd_amd as sgc
import lm_ref
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 37, 4099])
@pytest.mark.parametrize("cols", [511, 512, 513, 516, 600, 650, 767, 768, 769, 772])
def test_widths_of_one_wave_and_two(rows, cols):
    announce(f"norm {rows}x{cols} fp32")
    g = torch.Generator().manual_seed(rows + cols)
    x, dy = torch.randn(rows, cols, generator=g) * 1.5 + 0.5, torch.randn(rows, cols, generator=g)
    w, b = torch.randn(cols, generator=g), torch.randn(cols, generator=g)
    r = sgc.layer_norm(x.cuda(), w.cuda(), b.cuda())
    for got, ref, tol, what in zip((r.y, r.mean, r.rstd), *lm_ref.norm(x, w, b, 1e-5), ("y", "mean", "rstd")):
        lm_ref.close(got, ref, tol, what)
    # a workspace of the size that the call asks for, between guards
    need = sgc.layer_norm_backward_workspace_bytes(rows, cols)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    gr = sgc.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), r.mean, r.rstd, ws=buf[256:256 + need])
    assert (buf[:256] == 0x5A).all() and (buf[256 + need:] == 0x5A).all()
    for got, ref, tol, what in zip((gr.dx, gr.dweight, gr.dbias), *lm_ref.norm_backward(dy, x, w, r.mean, r.rstd),
                                   ("dx", "dweight", "dbias")):
        lm_ref.close(got, ref, tol, what)
