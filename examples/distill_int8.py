"""Trains a low-precision student by distillation, data-parallel, on one GPU.

The student is one output layer whose weight is held in 8 bits for its products
(a real copy takes the updates). Each step, each of a few workers
  - runs its batch through the 8-bit layer,
  - takes loss and gradient against the teacher's top logits,
  - takes the 8-bit layer's weight gradient (fp32),
  - encodes it as a QSGD stream, which is what workers send each other;
then the streams are decoded and summed into one gradient, and the weight is
updated and quantized again. The data is synthetic: the teacher is a random layer.

    python examples/distill_int8.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_sgd_amd as q  # noqa: E402


def train(steps=60, workers=2, batch=256, width=512, vocab=8192, top=32, lr=20.0, levels=64, bucket=4096, seed=0,
          report=lambda *a: None):
    """Returns each step's mean loss and the bits a coordinate that the streams took."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher = torch.randn(vocab, width, generator=g, device="cuda") * (3.0 / width ** 0.5)
    weight = torch.zeros(vocab, width, device="cuda")
    weight.normal_(std=0.2 / width ** 0.5, generator=g)
    share = torch.full((batch,), 1.0 / (batch * workers), device="cuda")
    losses, bits = [], 0
    for step in range(steps):
        w, sw = q.int8_quantize(weight)
        words, offsets, counts, loss = [], [], [], 0.0
        for worker in range(workers):
            x = torch.randn(batch, width, generator=g, device="cuda").bfloat16()
            said = x.float() @ teacher.t()
            t, idx = said.topk(top, dim=1)
            lse = torch.logsumexp(said, dim=1)
            y, xq, sx = q.int8_linear(x, w, sw, keep=True)
            row, dz = q.distill_topk_step(y, idx, t, share, teacher_lse=lse, out=y)  # the gradient in the logits' place
            _, gw = q.int8_linear_backward(dz, xq, sx, w, sw, need_gx=False)
            stream, count, starts = q.encode(gw.view(-1), levels, bucket, seed=step * workers + worker)
            words.append(stream)
            offsets.append(starts)
            counts.append(count)
            loss = loss + (row * share).sum()
        total = torch.zeros(vocab * width, device="cuda")
        q.decode_accumulate(words, offsets, total.numel(), levels, bucket, total)
        weight.sub_(total.view(vocab, width), alpha=lr)
        losses.append(float(loss))
        bits += sum(int(c) for c in counts)
        report(step, losses[-1])
    return losses, bits / (steps * workers * vocab * width)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    losses, bits = train(a.steps, report=lambda i, v: print(f"step {i}: loss {v:.4f}", flush=True) if i % 10 == 0 else None)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; {bits:.3f} bits a gradient coordinate")


if __name__ == "__main__":
    main()
