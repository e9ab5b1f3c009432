"""Training a small language model, and a student from its top logits.

The model: a tied embedding, pre-norm blocks x + W2 gelu(W1 norm(x) + b1) + b2,
a last norm, and the embedding again as the head.  The products with their
bias, activation and residual are linear_forward and linear_backward, the loss
never keeps its logits (linear_cross_entropy_*), gradients add up over
micro-batches in the tensors that the list step reads.  Then a narrower student
learns from the teacher's best logits only (distill_*).

    python examples/language_model.py [--steps N] [--dim D]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import optimizer_step_resumable_gb300 as osr  # noqa: E402

MICRO = 2  # micro-batches a step


class Model:
    """Parameters in the list's order: the embedding, then gain, shift, w1, b1,
    w2, b2 of each block, then the last gain and shift.  w1 is stored (in, out),
    as is w2."""

    def __init__(self, vocab, dim, blocks, seed=0):
        r = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sigma):
            return torch.empty(shape, device="cuda").normal_(0, sigma, generator=r)

        self.vocab, self.dim, self.blocks, self.wide = vocab, dim, blocks, 4 * dim
        self.w = [normal(vocab, dim, sigma=0.1)]
        for _ in range(blocks):
            self.w += [torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda"),
                       normal(dim, self.wide, sigma=dim ** -0.5),
                       torch.zeros(self.wide, device="cuda"),
                       normal(self.wide, dim, sigma=0.5 * self.wide ** -0.5),
                       torch.zeros(dim, device="cuda")]
        self.w += [torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda")]
        self.g = [torch.zeros_like(w) for w in self.w]
        self.copy = [w.bfloat16() for w in self.w]  # what the passes read
        m, v = ([torch.zeros_like(w) for w in self.w] for _ in range(2))
        self.list = osr.adamw_list_create(self.w, self.g, m, v, w_lp=self.copy,
                                          decay=[w.dim() == 2 for w in self.w])
        self.norm = osr.layernorm_create(dim)
        self.up = osr.linear_create(dim, self.wide)
        self.down = osr.linear_create(self.wide, dim)
        self.head = osr.linear_create(dim, vocab)
        self.loss = osr.linear_cross_entropy_create(dim, vocab)

    def close(self):
        for x in (self.list, self.norm, self.up, self.down, self.head, self.loss):
            x.close()

    def forward(self, tokens):
        """The last norm's output, and what the backward pass needs."""
        x = self.copy[0][tokens]
        saved = []
        for k in range(self.blocks):
            gain, shift, w1, b1, w2, b2 = self.copy[1 + 6 * k:7 + 6 * k]
            y, mean, rstd = osr.layernorm_forward(self.norm, x, gain, shift)
            z = torch.empty(len(tokens), self.wide, device="cuda", dtype=torch.bfloat16)
            h = osr.linear_forward(self.up, y, w1.T, b1, activation="gelu", z=z)
            saved.append((x, y, mean, rstd, z, h))
            x = osr.linear_forward(self.down, h, w2.T, b2, residual=x)
        y, mean, rstd = osr.layernorm_forward(self.norm, x, *self.copy[-2:])
        return y, (tokens, saved, x, mean, rstd)

    def backward(self, dy, state):
        """Adds the gradients of everything below the head to self.g."""
        tokens, saved, x, mean, rstd = state
        dx, _, _ = osr.layernorm_backward(self.norm, dy, x, self.copy[-2], mean, rstd,
                                          dweight=self.g[-2], dbias=self.g[-1], accumulate=True)
        for k in reversed(range(self.blocks)):
            gain, _, w1, _, w2, _ = self.copy[1 + 6 * k:7 + 6 * k]
            d_gain, d_shift, d_w1, d_b1, d_w2, d_b2 = self.g[1 + 6 * k:7 + 6 * k]
            x, y, mean, rstd, z, h = saved[k]
            dh, _, _ = osr.linear_backward(self.down, dx, h, w2.T, dweight=d_w2.T, dbias=d_b2,
                                           accumulate=True)
            d_norm, _, _ = osr.linear_backward(self.up, dh, y, w1.T, z=z, activation="gelu",
                                               dweight=d_w1.T, dbias=d_b1, accumulate=True)
            below, _, _ = osr.layernorm_backward(self.norm, d_norm, x, gain, mean, rstd,
                                                 dweight=d_gain, dbias=d_shift, accumulate=True)
            dx = dx + below
        self.g[0].index_add_(0, tokens, dx.float())

    def learn(self, tokens, target):
        """Adds the gradients of the targets' mean cross entropy; the rows' losses."""
        y, state = self.forward(tokens)
        loss, lse = osr.linear_cross_entropy_forward(self.loss, y, self.copy[0], target)
        dy, _ = osr.linear_cross_entropy_backward(self.loss, y, self.copy[0], target, lse,
                                                  scale=1.0 / len(tokens), dweight=self.g[0],
                                                  accumulate=True)
        self.backward(dy, state)
        return loss

    def logits(self, y):
        return osr.linear_forward(self.head, y, self.copy[0])

    def learn_from(self, tokens, ids, values, temperature):
        """The same against a teacher's best logits."""
        y, state = self.forward(tokens)
        logits = self.logits(y)
        with osr.distill_create(self.vocab, ids.shape[-1]) as ds:
            loss, lse = osr.distill_forward(ds, logits, ids, values, temperature=temperature)
            dl = osr.distill_backward(ds, logits, ids, values, lse, temperature=temperature,
                                      scale=1.0 / len(tokens), dlogits=logits)
        dy, _, _ = osr.linear_backward(self.head, dl, y, self.copy[0], dweight=self.g[0],
                                       accumulate=True)
        self.backward(dy, state)
        return loss

    def step(self, t):
        osr.adamw_list_step(self.list, t, lr=2e-3, wd=0.01, clip=1.0, grad_scale=1.0 / MICRO,
                            zero_grad=True)


def batch(vocab, rows, t, i):
    """Tokens, and as each one's target the next of a fixed cycle; every tenth row
    is padding."""
    r = torch.Generator(device="cuda").manual_seed(1000 * t + i)
    tokens = torch.randint(0, vocab, (rows,), device="cuda", generator=r)
    target = (tokens * 7 + 3) % vocab
    target[::10] = -100
    return tokens, target


def main(steps=100, dim=128, vocab=1000, blocks=2, rows=1024, k=16, temperature=2.0):
    """(the teacher's mean losses, the student's)."""
    teacher, student = Model(vocab, dim, blocks), Model(vocab, max(32, dim // 2), 1, seed=1)
    told = []
    for t in range(1, steps + 1):
        losses = [teacher.learn(*batch(vocab, rows, t, i)) for i in range(MICRO)]
        teacher.step(t)
        told.append(float(torch.cat(losses).mean()))
    norm, _ = osr.adamw_list_last_norm(teacher.list)  # raises NonFiniteGradient
    heard = []
    for t in range(1, steps + 1):
        losses = []
        for i in range(MICRO):
            tokens, _ = batch(vocab, rows, t, i)
            best = teacher.logits(teacher.forward(tokens)[0]).topk(k, dim=1)
            losses.append(student.learn_from(tokens, best.indices, best.values, temperature))
        student.step(t)
        heard.append(float(torch.cat(losses).mean()))
    osr.adamw_list_last_norm(student.list)
    print(f"teacher: loss {told[0]:.4f} -> {told[-1]:.4f}, last gradient norm {norm:.4f}; "
          f"student: {heard[0]:.4f} -> {heard[-1]:.4f}")
    teacher.close()
    student.close()
    return told, heard


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=100)
    p.add_argument("--dim", type=int, default=128)
    a = p.parse_args()
    main(steps=a.steps, dim=a.dim)
