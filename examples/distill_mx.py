"""Data-parallel distillation in 4 bits: a student learns a teacher's next-token distribution with
its layers' products on microscaled 4-bit operands, and the workers' gradients are exchanged as
Global-QSGD codes.

    python examples/distill_mx.py [--steps 30] [--workers 4] [--tokens 512] [--vocab 4096]

One step: the teacher's logits -> gq.token_logprobs (its 32 most likely tokens, with the rest as
one bucket) -> per worker, two lm.mx_linear layers, lm.distill and their gradients ->
gq.global_norm and gq.fused_mean over the workers' gradients (8-bit codes, int16 sums) -> Adam on
the fp32 master weights.  The workers' data is synthetic; they share one GPU.
"""
import argparse
import itertools
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from allreduce_compatible_gradient_amd import gq, lm  # noqa: E402


def run(steps=30, workers=4, tokens=512, width=256, hidden=512, vocab=4096, top=32, seed=1,
        lr=2e-3, say=print):
    """Trains the student; returns the mean loss of every step and the teacher's mean entropy."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    t1, t2 = normal(hidden, width) / width ** 0.5, normal(vocab, hidden) * 2.5 / hidden ** 0.5
    w1 = (normal(hidden, width) / width ** 0.5).requires_grad_()
    w2 = (normal(vocab, hidden) * 0.02).requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=lr)
    sizes = [w1.numel(), w2.numel()]
    losses, entropy = [], 0.0
    seeds = itertools.count(seed)   # every rounding of every step draws with a seed of its own
    for step in range(steps):
        flat, mean_loss = [], 0.0
        for k in range(workers):
            x = normal(tokens, width).to(torch.bfloat16)
            teacher = torch.relu(x.float() @ t1.T) @ t2.T
            sampled = torch.zeros(tokens, dtype=torch.int64, device="cuda")
            _, h, ids, lps = gq.token_logprobs(teacher, sampled, top=top)
            y = torch.relu(lm.mx_linear(x, w1, seed=next(seeds), worker=k))
            logits = lm.mx_linear(y, w2, seed=next(seeds), worker=k)
            loss = lm.distill(logits, ids, lps, tail=True).mean()
            grads = torch.autograd.grad(loss, (w1, w2))
            flat.append(torch.cat([d.reshape(-1) for d in grads]))
            mean_loss += float(loss.detach()) / workers
            entropy += float(h.mean()) / (workers * steps)
        # the exchange: one scale a layer, codes that add, one decode
        offsets = [0, sizes[0], sizes[0] + sizes[1]]
        scale, _ = gq.global_norm(flat, offsets)
        mean = gq.fused_mean(flat, scale, gq.UNIFORM, 127, 8, seed=next(seeds), acc_bits=16,
                             offsets=offsets)
        for w, d in zip((w1, w2), mean.split(sizes)):
            w.grad = d.view_as(w)
        opt.step()
        losses.append(mean_loss)
        if say and (step % 10 == 0 or step == steps - 1):
            say("step %3d  distillation loss %.4f" % (step, mean_loss))
    return losses, entropy


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 30), ("workers", 4), ("tokens", 512), ("vocab", 4096)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    losses, entropy = run(a.steps, a.workers, a.tokens, vocab=a.vocab)
    print("loss %.4f -> %.4f (the teacher's entropy: %.3f)" % (losses[0], losses[-1], entropy))
