"""Trains an output head as a policy: its tokens are sampled and rewarded, and its weight is updated by the preconditioner.

A layer norm with weight and bias, then logits = y W^T in 8 bits.  One step samples a token for every hidden state, scores
it, and takes a few updates on those samples:

    precond_layer_norm        h + r, the norm, its 8-bit form, mean and 1 / std
    precond_quantize8         W in 128 x 128 blocks (both orientations)
    precond_gemm8             logits = y W^T
    precond_policy            (sampling) the taken tokens' log probabilities, under this policy and the reference
    precond_policy            (updates) the clipped loss with a KL term, and dlogits, in place
    precond_quantize8         dlogits by rows and by columns, y by columns
    precond_gemm8             dy = dlogits W, and G = dlogits^T y in fp32
    precond_layer_norm_grad   the gradients of the stream, of the norm's weight and of its bias
    precond_clip_grads        all of the head's gradients scaled down to a largest norm
    precond_step              U = L^-1/4 G R^-1/4 from the Gram EMAs of G

and W -= lr U.  Run it on a GPU: python examples/policy_head.py [--steps N]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import shampoo_roots_gb300 as sr  # noqa: E402

EPS = 1e-5


class PolicyHead:
    """The head's weight, the norm's weight and bias, the optimizer state and the buffers of a step."""

    def __init__(self, tokens: int, d: int, vocab: int, lr: float = 0.02, tau: float = 1.0, kl: float = 0.02, max_norm: float = 0.1,
                 seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.tokens, self.d, self.vocab, self.lr, self.tau, self.kl, self.max_norm = tokens, d, vocab, lr, tau, kl, max_norm
        self.pc = sr.Preconditioner(torch.cuda.current_device())
        self.W = torch.randn(vocab, d, generator=g, device="cuda") * d ** -0.5 * 0.3
        self.w, self.b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
        self.L, self.R = (torch.zeros(n, n, device="cuda") for n in (vocab, d))
        self.h = torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda")
        self.mean, self.rstd = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.y, self.yt = sr.empty8(tokens, d), sr.empty8(d, tokens)
        self.W8, self.Wt8 = sr.empty8(vocab, d), sr.empty8(d, vocab)
        self.logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device="cuda")
        self.dl, self.dlt = sr.empty8(tokens, vocab), sr.empty8(vocab, tokens)
        self.dy, self.dx = (torch.empty(tokens, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.dw, self.db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        self.G, self.U = (torch.empty(vocab, d, device="cuda") for _ in range(2))
        self.loss, self.logp = (torch.empty(tokens, device="cuda") for _ in range(2))
        self.norm = torch.empty((), device="cuda")
        self.grads = sr.TensorList([self.G, self.dw, self.db])      # the buffers stay, so the list does

    def forward(self, x, r):
        """The logits of a batch; the norm's outputs are left in the object."""
        h = self.pc.h
        sr.precond_layer_norm(h, x, self.w, EPS, bias=self.b, residual=r, total=self.h, q=self.y[0], scale=self.y[1], mean=self.mean,
                              rstd=self.rstd)
        sr.precond_quantize8(h, self.W, *self.W8, *self.Wt8, block=sr.BLOCK_TILE)
        sr.precond_gemm8(h, *self.y, *self.W8, self.logits)
        return self.logits

    def score(self, x, r, ids, out):
        """The taken tokens' log probabilities under this policy."""
        sr.precond_policy(self.pc.h, self.forward(x, r), ids, temperature=self.tau, logp=out)
        return out

    def gradients(self, x, r, ids, advantage, old, ref, weight):
        """Loss of every token; G, dw, db and dx are left in the object."""
        h = self.pc.h
        self.forward(x, r)
        sr.precond_policy(h, self.logits, ids, advantage=advantage, old_logp=old, ref_logp=ref, weight=weight, temperature=self.tau,
                          kl=self.kl, loss=self.loss, logp=self.logp, dlogits=self.logits)
        sr.precond_quantize8(h, self.logits, *self.dl, *self.dlt)
        sr.precond_quantize8(h, self.y[0], qt=self.yt[0], scale_t=self.yt[1], x_scale=self.y[1])
        sr.precond_gemm8(h, *self.dl, *self.Wt8, self.dy)
        sr.precond_gemm8(h, *self.dlt, *self.yt, self.G)
        sr.precond_layer_norm_grad(h, self.dy, self.h, self.w, self.mean, self.rstd, self.dx, self.dw, db=self.db)
        return self.loss

    def update(self):
        """Clips the gradients and moves the weights."""
        sr.precond_clip_grads(self.pc.h, self.grads, self.max_norm, self.norm)
        sr.precond_step(self.pc.h, [self.G], [self.L], [self.R], 0.95, 1e-4, -0.25, out=[self.U])
        self.W.sub_(self.U, alpha=self.lr * (self.W.numel() ** 0.5) / float(self.U.norm().clamp(min=1e-30)))
        self.w.sub_(self.dw, alpha=self.lr)
        self.b.sub_(self.db, alpha=self.lr)


def batch(tokens, d, gen):
    """Hidden states, a residual, and the tokens' weights (one in eight is a prompt's)."""
    x, r = (torch.randn(tokens, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    live = (torch.rand(tokens, generator=gen, device="cuda") > 0.125).float()
    return x, r, live / live.sum().clamp(min=1)


def sample(logits, tau, gen):
    noise = torch.empty(logits.shape, device=logits.device).exponential_(generator=gen)
    return (torch.softmax(logits.float() / tau, dim=1) / noise).argmax(dim=1)


def main(steps: int = 20, tokens: int = 2000, d: int = 256, vocab: int = 300, epochs: int = 2, verbose: bool = True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    wanted = torch.randn(vocab, d, generator=gen, device="cuda")          # a token is worth how well it suits the state
    head, reference = PolicyHead(tokens, d, vocab), PolicyHead(tokens, d, vocab)
    old, ref = (torch.empty(tokens, device="cuda") for _ in range(2))
    rewards = []
    for i in range(steps):
        x, r, weight = batch(tokens, d, gen)
        ids = sample(head.forward(x, r), head.tau, gen)
        head.score(x, r, ids, old)
        reference.score(x, r, ids, ref)
        reward = torch.tanh((head.h.float() * wanted[ids]).sum(dim=1) / d ** 0.5)
        advantage = (reward - reward.mean()) / reward.std().clamp(min=1e-6)
        for _ in range(epochs):
            loss = head.gradients(x, r, ids, advantage, old, ref, weight).sum()
            head.update()
        rewards.append(float(reward.mean()))
        if verbose and (i % 5 == 0 or i == steps - 1):
            print(f"step {i:3d}  reward {rewards[-1]:+.4f}  loss {float(loss):+.4f}  gradient norm {float(head.norm):.4f}")
    return rewards


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    main(ap.parse_args().steps)
