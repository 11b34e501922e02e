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

With --bits 8 the model is an RMS norm's, and what lies between the norm and
the loss is in 8 bits: the teacher is a network of its own, whose normed rows
and head are 8-bit integers (rms_norm_q8, int8_linear), and the student keeps
its norm's input in 8 bits for the backward pass (quantize_q8,
rms_norm_backward_q8), which gives the normed rows again for the head's
gradient.

    python examples/distill_lm.py [--vocab 98] [--width 512] [--steps 60] [--bits 8]
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


@dataclass
class Student8(Student):
    """The student with an RMS norm, whose input is all that is kept of it: in 8 bits."""

    def logits(self, tokens: torch.Tensor):
        x = self.part(self.flat, 0)[tokens].bfloat16()
        n = sgc.rms_norm(x, self.part(self.flat, 1))
        return n.y @ self.part(self.flat, 3).bfloat16().t(), (sgc.quantize_q8(x, group=64), n.rstd)

    def gradient(self, tokens: torch.Tensor, saved, dlogits: torch.Tensor, out: torch.Tensor) -> None:
        kept, rstd = saved
        dy = dlogits @ self.part(self.flat, 3).bfloat16()
        g = sgc.rms_norm_backward_q8(dy, kept, self.part(self.flat, 1), rstd, dx=dy, dweight=self.part(out, 1),
                                     want_y=True)
        self.part(out, 2).zero_()  # an RMS norm has no bias
        self.part(out, 3).copy_(dlogits.t() @ g.y)
        self.part(out, 0).zero_().index_add_(0, tokens, g.dx.float())


@dataclass
class Teacher8:
    """Embedding, RMS norm and head of a fixed network; it scores in 8-bit integers."""
    embedding: torch.Tensor
    weight: torch.Tensor
    head: sgc.Quantized

    @classmethod
    def make(cls, vocab: int, width: int, gen: torch.Generator) -> "Teacher8":
        normal = lambda *s: torch.empty(*s, device="cuda").normal_(0.0, 1.0, generator=gen)  # noqa: E731
        return cls(normal(vocab, width).bfloat16(), 1.0 + 0.1 * normal(width),
                   sgc.quantize_q8(normal(vocab, width) * (2.0 * width ** -0.5), group=0))

    def logits(self, tokens: torch.Tensor) -> torch.Tensor:
        return sgc.int8_linear(sgc.rms_norm_q8(self.embedding[tokens], self.weight).q8, self.head)


def train(vocab: int = 98, width: int = 512, rows: int = 1024, steps: int = 60, workers: int = 4, top: int = 16,
          keep_ppm: int = 50000, scale: float = 1.0, lr: float = 4.0, seed: int = 0, bits: int = 16,
          log=print):
    """Teaches a student; its mean divergence before and after, and the bits sent per parameter and step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if bits == 8:
        score = Teacher8.make(vocab, width, gen).logits
        student = Student8.make(vocab, width, gen)
    else:
        teacher = torch.empty(vocab, vocab, device="cuda").normal_(0.0, 2.0, generator=gen)  # next-token logits
        score = teacher.__getitem__
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
        t = sgc.token_logprobs(score(tokens), scale=scale, top=top)
        z, _ = student.logits(tokens)
        return float(sgc.distill(z, t.top_idx, t.top_logp, mode=sgc.DISTILL_TAIL, scale=scale).loss.mean())

    first, sent = divergence(), 0
    for step in range(steps):
        messages = []
        for w in range(workers):
            tokens = draw()
            t = sgc.token_logprobs(score(tokens), scale=scale, top=top)
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
    p.add_argument("--bits", type=int, choices=(8, 16), default=16)
    a = p.parse_args()
    first, last, bits = train(a.vocab, a.width, a.rows, a.steps, a.workers, a.top, a.keep_ppm,
                              bits=a.bits)
    print(f"divergence from the teacher {first:.4f} -> {last:.4f}, {bits:.2f} bits sent per parameter and step")


if __name__ == "__main__":
    main()
