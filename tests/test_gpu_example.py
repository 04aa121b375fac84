"""examples/distilled_head.py on the GPU: the step's gradients against a plain 64-bit backward pass, and training."""
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


def test_gradients():
    """Each result against 64 bits on what the step itself holds before it (8-bit values, bf16 logits), so that only
    the rounding of that result remains; and G against the backward pass of the unrounded step."""
    import distilled_head as dh
    import shampoo_roots_gb300 as sr
    head = dh.DistilledHead(333, 200, 450, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    teacher_W = torch.randn(450, 200, generator=gen, device="cuda") * 3 * 200 ** -0.5
    x, r, ids, t, w = dh.batch(teacher_W, 333, 200, 16, head.tau, gen)
    loss = head.gradients(x, r, ids, t, w)
    # fp32 sums of exact products: 1e-6; bf16 results: 2^-8
    G = sr.dequantize8(*head.dlt).double() @ sr.dequantize8(*head.yt).double().t()
    assert rel(head.G, G) <= 2e-6
    dy = sr.dequantize8(*head.dl).double() @ sr.dequantize8(*head.Wt8).double().t()
    assert rel(head.dy, dy) <= 2 ** -8
    # y by columns is y by rows, but for values below a block's smallest number
    y = sr.dequantize8(*head.y)
    assert rel(sr.dequantize8(*head.yt).t(), y) <= 1e-3
    # the same step in 64 bits throughout; 8-bit rounding of y, W and dlogits is 2^-4 a value at most, about 2.6 % in norm
    h = (x.float() + r.float()).bfloat16().double().requires_grad_()
    W = head.W.double().requires_grad_()
    n = h / torch.sqrt(h.square().mean(1, keepdim=True) + dh.EPS)
    logq = torch.log_softmax(n @ W.t() / head.tau, 1).gather(1, ids)
    logp = torch.log_softmax(t.double() / head.tau, 1)
    want = head.tau ** 2 * w.double() * (logp.exp() * (logp - logq)).sum(1)
    want.sum().backward()
    assert rel(loss, want) <= 2e-2
    assert rel(head.G, W.grad) <= 0.06
    assert rel(head.dx, h.grad) <= 0.06


def test_training():
    import distilled_head as dh
    losses = dh.main(steps=30, verbose=False)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] <= 0.6 * losses[0], losses
