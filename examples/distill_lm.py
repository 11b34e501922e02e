"""A student language model taught from a teacher's top entries, its gradients
sparsified and exchanged: the operators of the loss end and the compression
path as a training step uses them together.

Several simulated workers share the student (embedding, layer norm, output
head) and teach it a fixed teacher's next-token distributions.  A step of one
worker:

    layer_norm -> logits -> (teacher: token_logprobs' top list) -> distill,
    loss and gradient in one call, the gradient in the logits' own place ->
    the head's and the norm's gradients; layer_norm_backward puts the weight's
    and bias' sums straight into their segments of the flat gradient ->
    compress against the worker's residual -> Rice code

and the receiver adds the workers' messages into one dense update.

    python examples/distill_lm.py [--vocab 98] [--width 512] [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compressed_sgd_amd as sgc  # noqa: E402


@dataclass
class Student:
    """Parameters as segments of one flat fp32 vector: what a layout describes."""
    vocab: int
    width: int
    flat: torch.Tensor
    layout: sgc.Layout

    @classmethod
    def make(cls, vocab: int, width: int, gen: torch.Generator) -> "Student":
        layout = sgc.Layout([vocab * width, width, width, vocab * width])
        s = cls(vocab, width, torch.empty(layout.n, device="cuda").normal_(0.0, width ** -0.5, generator=gen), layout)
        s.part(s.flat, 0).normal_(0.0, 1.0, generator=gen)
        s.part(s.flat, 1).fill_(1.0)
        s.part(s.flat, 2).zero_()
        return s

    def part(self, flat: torch.Tensor, k: int) -> torch.Tensor:
        a, b = self.layout.seg_off[k], self.layout.seg_off[k + 1]
        return flat[a:b].view(self.vocab, self.width) if k in (0, 3) else flat[a:b]

    def logits(self, tokens: torch.Tensor):
        """Logits in bf16, and what the backward pass needs."""
        x = self.part(self.flat, 0)[tokens]
        n = sgc.layer_norm(x, self.part(self.flat, 1), self.part(self.flat, 2))
        y = n.y.bfloat16()
        return y @ self.part(self.flat, 3).bfloat16().t(), (x, n, y)

    def gradient(self, tokens: torch.Tensor, saved, dlogits: torch.Tensor, out: torch.Tensor) -> None:
        """The flat gradient (written over `out`) from that of the logits."""
        x, n, y = saved
        self.part(out, 3).copy_(dlogits.t() @ y)
        dy = (dlogits @ self.part(self.flat, 3).bfloat16()).float()
        g = sgc.layer_norm_backward(dy, x, self.part(self.flat, 1), n.mean, n.rstd, dx=dy,
                                    dweight=self.part(out, 1), dbias=self.part(out, 2))
        self.part(out, 0).zero_().index_add_(0, tokens, g.dx)


def train(vocab: int = 98, width: int = 512, rows: int = 1024, steps: int = 60, workers: int = 4, top: int = 16,
          keep_ppm: int = 50000, scale: float = 1.0, lr: float = 4.0, seed: int = 0, log=print):
    """Teaches a student; its mean divergence before and after, and the bits sent per parameter and step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    teacher = torch.empty(vocab, vocab, device="cuda").normal_(0.0, 2.0, generator=gen)  # next-token logits
    student = Student.make(vocab, width, gen)
    layout = student.layout
    residual = [torch.zeros(layout.n, device="cuda") for _ in range(workers)]
    grad = torch.empty(layout.n, device="cuda")
    update = torch.empty(layout.n, device="cuda")
    weight = torch.full((rows,), 1.0 / rows, device="cuda")  # the rows' upstream gradients: a mean
    b = sgc.rice_param(keep_ppm / 1e6)

    def draw():
        return torch.randint(0, vocab, (rows,), device="cuda", generator=gen)

    def divergence() -> float:
        tokens = torch.arange(vocab, device="cuda")
        t = sgc.token_logprobs(teacher, scale=scale, top=top)
        z, _ = student.logits(tokens)
        return float(sgc.distill(z, t.top_idx, t.top_logp, mode=sgc.DISTILL_TAIL, scale=scale).loss.mean())

    first, sent = divergence(), 0
    for step in range(steps):
        messages = []
        for w in range(workers):
            tokens = draw()
            t = sgc.token_logprobs(teacher[tokens], scale=scale, top=top)
            z, saved = student.logits(tokens)
            d = sgc.distill(z, t.top_idx, t.top_logp, mode=sgc.DISTILL_TAIL, scale=scale, dloss=weight, dlogits=z)
            student.gradient(tokens, saved, d.dlogits, grad)
            comp = sgc.compress(layout, grad, residual[w], keep_ppm=keep_ppm)
            enc = sgc.encode(layout, comp.idx, comp.counts, comp.cap, b=b)
            messages.append(sgc.golomb_message(comp, enc))
            sent += 32 * comp.cap + int(enc.nbits[0])
        sgc.decode_accumulate(layout, messages, update)
        student.flat.sub_(update, alpha=lr / workers)
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step}: loss {float(d.loss.mean()):.4f}")
    last = divergence()
    return first, last, sent / (steps * workers * layout.n)


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--vocab", type=int, default=98)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--rows", type=int, default=1024)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--workers", type=int, default=4)
    p.add_argument("--top", type=int, default=16)
    p.add_argument("--keep-ppm", type=int, default=50000)
    a = p.parse_args()
    first, last, bits = train(a.vocab, a.width, a.rows, a.steps, a.workers, a.top, a.keep_ppm)
    print(f"divergence from the teacher {first:.4f} -> {last:.4f}, {bits:.2f} bits sent per parameter and step")


if __name__ == "__main__":
    main()
