"""Distils an output head whose weight is multiplied in 8 bits and updated by the preconditioner.

A teacher's top logits for a batch of hidden states teach a student head: RMS norm, then logits = y W^T.  One step is

    precond_rms_norm        h + r, the norm, its 8-bit form, 1 / rms
    precond_quantize8       W in 128 x 128 blocks (both orientations)
    precond_gemm8           logits = y W^T
    precond_distill         the loss and dlogits, in place
    precond_quantize8       dlogits by rows and by columns, y by columns
    precond_gemm8           dy = dlogits W, and G = dlogits^T y in fp32
    precond_rms_norm_grad   the gradients of the stream and of the norm's weight
    precond_step            U = L^-1/4 G R^-1/4 from the Gram EMAs of G

and W -= lr U.  Run it on a GPU: python examples/distilled_head.py [--steps N]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import shampoo_roots_gb300 as sr  # noqa: E402

EPS = 1e-6


class DistilledHead:
    """The head's weight, the norm's weight, the optimizer state and the buffers of a step."""

    def __init__(self, tokens: int, d: int, vocab: int, lr: float = 0.02, tau: float = 2.0, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.tokens, self.d, self.vocab, self.lr, self.tau = tokens, d, vocab, lr, tau
        self.pc = sr.Preconditioner(torch.cuda.current_device())
        self.W = torch.randn(vocab, d, generator=g, device="cuda") * d ** -0.5 * 0.1
        self.w = torch.ones(d, device="cuda")
        self.L, self.R = (torch.zeros(n, n, device="cuda") for n in (vocab, d))
        self.h = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda")
        self.rstd = torch.empty(tokens, device="cuda")
        self.y, self.yt = sr.empty8(tokens, d), sr.empty8(d, tokens)
        self.W8, self.Wt8 = sr.empty8(vocab, d), sr.empty8(d, vocab)
        self.logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device="cuda")
        self.dl, self.dlt = sr.empty8(tokens, vocab), sr.empty8(vocab, tokens)
        self.dy, self.dx = (torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.dw = torch.empty(d, device="cuda")
        self.G, self.U = (torch.empty(vocab, d, device="cuda") for _ in range(2))
        self.loss = torch.empty(tokens, device="cuda")

    def gradients(self, x, r, ids, teacher, weight):
        """Loss of every token; G, dw and dx are left in the object."""
        h = self.pc.h
        sr.precond_rms_norm(h, x, self.w, EPS, residual=r, total=self.h, q=self.y[0], scale=self.y[1], rstd=self.rstd)
        sr.precond_quantize8(h, self.W, *self.W8, *self.Wt8, block=sr.BLOCK_TILE)
        sr.precond_gemm8(h, *self.y, *self.W8, self.logits)
        sr.precond_distill(h, self.logits, ids, teacher, self.loss, weight=weight, temperature=self.tau, dlogits=self.logits)
        sr.precond_quantize8(h, self.logits, *self.dl, *self.dlt)
        sr.precond_quantize8(h, self.y[0], qt=self.yt[0], scale_t=self.yt[1], x_scale=self.y[1])
        sr.precond_gemm8(h, *self.dl, *self.Wt8, self.dy)
        sr.precond_gemm8(h, *self.dlt, *self.yt, self.G)
        sr.precond_rms_norm_grad(h, self.dy, self.h, self.w, self.rstd, self.dx, self.dw)
        return self.loss

    def step(self, x, r, ids, teacher, weight):
        loss = self.gradients(x, r, ids, teacher, weight).sum()
        sr.precond_step(self.pc.h, [self.G], [self.L], [self.R], 0.95, 1e-4, -0.25, out=[self.U])
        self.W.sub_(self.U, alpha=self.lr * (self.W.numel() ** 0.5) / float(self.U.norm().clamp(min=1e-30)))
        self.w.sub_(self.dw, alpha=self.lr)
        return float(loss)


def batch(teacher_W, tokens, d, top, tau, gen):
    """Hidden states, a residual, the teacher's top logits and the tokens' weights (one in eight is padding)."""
    x, r = (torch.randn(tokens, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    f = x.float() + r.float()
    logits = (f * torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)) @ teacher_W.t()
    teacher, ids = torch.topk(logits, top, dim=1)
    live = (torch.rand(tokens, generator=gen, device="cuda") > 0.125).float()
    return x, r, ids, teacher.contiguous(), live / live.sum().clamp(min=1)


def main(steps: int = 40, tokens: int = 1000, d: int = 256, vocab: int = 700, top: int = 32, verbose: bool = True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    teacher_W = torch.randn(vocab, d, generator=gen, device="cuda") * 3 * d ** -0.5
    head = DistilledHead(tokens, d, vocab)
    losses = []
    for i in range(steps):
        losses.append(head.step(*batch(teacher_W, tokens, d, top, head.tau, gen)))
        if verbose and (i % 5 == 0 or i == steps - 1):
            print(f"step {i:3d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    main(ap.parse_args().steps)
