"""examples/policy_head.py on the GPU: the operators of a policy's step together, each against 64 bits on what the step
itself holds before it, the whole against a plain 64-bit backward pass, and the run."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def test_gradients_and_clipping():
    import policy_head as ph
    import shampoo_roots_gb300 as sr
    tokens, d, vocab = 333, 200, 450
    head = ph.PolicyHead(tokens, d, vocab, seed=3, tau=0.8, kl=0.1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    head.w.add_(0.2 * torch.randn(d, generator=gen, device="cuda"))
    head.b.add_(0.2 * torch.randn(d, generator=gen, device="cuda"))
    x, r, weight = ph.batch(tokens, d, gen)
    old, ref = (torch.empty(tokens, device="cuda") for _ in range(2))
    ids = ph.sample(head.forward(x, r), head.tau, gen)
    logits = head.logits.clone()
    head.score(x, r, ids, old)
    scored = torch.log_softmax(logits.double() / head.tau, 1).gather(1, ids[:, None])[:, 0]
    assert float((old.double() - scored).abs().max()) <= 1e-5          # fp32 sums of 450 powers, logits of a few units
    old -= 0.05
    ref.copy_(old + 0.3 * torch.randn(tokens, generator=gen, device="cuda"))
    advantage = torch.randn(tokens, generator=gen, device="cuda")
    loss = head.gradients(x, r, ids, advantage, old, ref, weight)
    # fp32 sums of exact products: 1e-6; bf16 results: 2^-8
    G = sr.dequantize8(*head.dlt).double() @ sr.dequantize8(*head.yt).double().t()
    assert rel(head.G, G) <= 2e-6
    # the same step in 64 bits throughout; 8-bit rounding of y, W and dlogits is 2^-4 a value at most, about 2.6 % in norm
    h = (x.float() + r.float()).bfloat16().double().requires_grad_()
    W, w, b = (t.double().requires_grad_() for t in (head.W, head.w, head.b))
    c = h - h.mean(1, keepdim=True)
    y = c / torch.sqrt(c.square().mean(1, keepdim=True) + ph.EPS) * w + b
    s = torch.log_softmax(y @ W.t() / head.tau, 1).gather(1, ids[:, None])[:, 0]
    # the step's log probabilities are those of 8-bit products: start from them, with the unrounded step's derivative
    s = s - s.detach() + head.logp.double()
    ratio, a = torch.exp(s - old.double()), advantage.double()
    e = ref.double() - s
    want = weight.double() * (-torch.minimum(ratio * a, ratio.clamp(0.8, 1.2) * a) + head.kl * (torch.exp(e) - e - 1))
    want.sum().backward()
    assert float((loss.double() - want.detach()).abs().max()) <= 1e-5 * float(want.detach().abs().max())
    for got, exact in ((head.G, W.grad), (head.dx, h.grad), (head.dw, w.grad), (head.db, b.grad)):
        assert rel(got, exact) <= 0.06
    # clipping: one factor for the three
    held = [t.clone() for t in head.grads.tensors]
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in held))
    head.max_norm = 0.25 * norm
    sr.precond_clip_grads(head.pc.h, head.grads, head.max_norm, head.norm)
    assert abs(float(head.norm) - norm) <= 2e-6 * norm
    for t, was in zip(head.grads.tensors, held):
        assert rel(t, 0.25 * was) <= 2e-6


def test_run():
    import policy_head as ph
    rewards = ph.main(steps=4, tokens=500, verbose=False)
    assert len(rewards) == 4 and all(math.isfinite(v) for v in rewards)
