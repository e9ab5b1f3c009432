"""Training with the layer norm and the list step: a stack of pre-norm
residual blocks x + W2 relu(W1 norm(x)), whose parameters live in tensors of
their own.  The matrices keep their Adam moments in 8 bits, the norms' gains
and shifts in 32; each step adds two micro-batches' gradients up, clips them
by their joint norm and updates everything in one call.  Half-way the state
is saved; a second run resumed from the file ends in the same bits.

    python examples/norm_and_list_step.py [--steps N] [--dim D] [--file PATH]
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
    """Parameters, gradients and moments, one tensor each, in the list's order."""

    def __init__(self, blocks, dim, seed=0):
        r = torch.Generator(device="cuda").manual_seed(seed)
        self.blocks, self.dim = blocks, dim
        self.w = []
        for _ in range(blocks):
            gain, shift = torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda")
            w1, w2 = (torch.empty(dim, dim, device="cuda").normal_(0, dim ** -0.5, generator=r)
                      for _ in range(2))
            self.w += [gain, shift, w1, w2]
        matrix = [w.dim() == 2 for w in self.w]
        self.g = [torch.zeros_like(w) for w in self.w]
        self.copy = [w.bfloat16() for w in self.w]  # what the forward pass reads
        self.m, self.v, self.ms, self.vs = [], [], [], []
        for w, eight in zip(self.w, matrix):
            for state, scale, kind in ((self.m, self.ms, torch.float8_e4m3fn),
                                       (self.v, self.vs, torch.float8_e5m2)):
                state.append(torch.zeros(w.shape, dtype=torch.uint8, device="cuda").view(kind)
                             if eight else torch.zeros_like(w))
                scale.append(torch.zeros(-(-w.numel() // osr.STATE_BLOCK), device="cuda")
                             if eight else None)
        self.norm = osr.layernorm_create(dim)
        # decay on the matrices, none on the norms
        self.list = osr.adamw_list_create(self.w, self.g, self.m, self.v, self.ms, self.vs,
                                          self.copy, decay=matrix)

    def state(self):
        return [self.w, self.m, self.v, self.ms, self.vs, self.copy]

    def close(self):
        self.list.close()
        self.norm.close()

    def forward_backward(self, x, target):
        """Adds the gradients of mean((f(x) - target)^2) to self.g; the loss."""
        saved = []
        for k in range(self.blocks):
            gain, shift, w1, w2 = self.copy[4 * k:4 * k + 4]
            y, mean, rstd = osr.layernorm_forward(self.norm, x, gain, shift)
            h = torch.relu(y @ w1)
            saved.append((x, y, mean, rstd, h))
            x = x + h @ w2
        diff = (x - target).float()
        dx = (diff * (2.0 / diff.numel())).bfloat16()
        for k in reversed(range(self.blocks)):
            gain, _, w1, w2 = self.copy[4 * k:4 * k + 4]
            d_gain, d_shift, d_w1, d_w2 = self.g[4 * k:4 * k + 4]
            xk, y, mean, rstd, h = saved[k]
            d_w2 += h.T @ dx
            dh = (dx @ w2.T) * (h > 0)
            d_w1 += y.T @ dh
            d_norm, _, _ = osr.layernorm_backward(self.norm, dh @ w1.T, xk, gain, mean, rstd,
                                                  dweight=d_gain, dbias=d_shift, accumulate=True)
            dx = dx + d_norm
        return float((diff * diff).mean())


def batch(t, i, rows, dim):
    """Micro-batch i of step t: a pure function of both, so a resumed run sees
    the batches that the first one saw."""
    r = torch.Generator(device="cuda").manual_seed(1000 * t + i)
    x = torch.empty(rows, dim, device="cuda").normal_(generator=r)
    return x.bfloat16(), torch.roll(x, 1, 1).bfloat16()


def train(model, first, last, rows):
    losses = []
    for t in range(first, last + 1):
        loss = sum(model.forward_backward(*batch(t, i, rows, model.dim)) for i in range(MICRO))
        osr.adamw_list_step(model.list, t, lr=1e-3, wd=0.01, clip=1.0, grad_scale=1.0 / MICRO,
                            seed=17, zero_grad=True)
        losses.append(loss / MICRO)
    return losses


def main(steps=200, dim=256, blocks=2, rows=512, path="norm_and_list_step.pt"):
    """Returns (losses, whether the resumed run ended in the same bits)."""
    half = steps // 2
    model = Model(blocks, dim)
    losses = train(model, 1, half, rows)
    torch.save({"step": half, "state": model.state()}, path)
    losses += train(model, half + 1, steps, rows)
    norm, factor = osr.adamw_list_last_norm(model.list)  # raises NonFiniteGradient

    again = Model(blocks, dim, seed=1)
    saved = torch.load(path)
    for mine, theirs in zip(again.state(), saved["state"]):
        for a, b in zip(mine, theirs):
            if a is not None:
                a.copy_(b)
    train(again, saved["step"] + 1, steps, rows)
    same = all(a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for p, q in zip(model.state(), again.state()) for a, b in zip(p, q))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}, last gradient norm {norm:.4f}, "
          f"clip factor {factor:.3f}, resumed run identical: {same}")
    model.close()
    again.close()
    return losses, same


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--dim", type=int, default=256)
    p.add_argument("--file", default="norm_and_list_step.pt")
    a = p.parse_args()
    main(steps=a.steps, dim=a.dim, path=a.file)
