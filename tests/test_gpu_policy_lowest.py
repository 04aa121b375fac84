"""Log probabilities of taken tokens far below the largest logit: masked with the type's lowest value they are finite
wherever fp32 holds them.  Tolerances as in test_gpu_policy.py."""
import math

import pytest
import torch

import shampoo_roots_gb300 as sr
from test_gpu_policy import E, inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu
MOST = torch.finfo(torch.float32).max


@pytest.mark.parametrize("tau", [0.7, 1.0, 4.0])
@pytest.mark.parametrize("rows,vocab,dtype", [(40, 700, "bf16"), (40, 700, "f32"), (200, 3001, "bf16"), (9, 40001, "bf16"), (200, 50001, "f32"),
                                              (4, 500003, "f32")])
def test_lowest(pc, rows, vocab, dtype, tau):  # noqa: F811
    z, ids, adv, old, _, weight = inputs(rows, vocab, dtype, 1.0)
    lowest = torch.finfo(z.dtype).min
    kind = torch.arange(rows) % 4
    at = torch.arange(rows)
    z[at[kind == 1], ids[kind == 1]] = lowest                        # the taken token forbidden
    z[kind == 2] = lowest                                            # everything forbidden but one
    z[at[kind == 2], (ids[kind == 2] + 1) % vocab] = 3.0
    z[kind == 3] = 0.5 * lowest                                      # beside the largest
    z[at[kind == 3], ids[kind == 3]] = lowest
    z[at[kind == 3], (ids[kind == 3] + 1) % vocab] = -lowest
    loss, logp, grad = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(z, device="cuda")
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=old.cuda(), weight=weight.cuda(), temperature=tau,
                      loss=loss, logp=logp, dlogits=grad)
    x = z.double() / tau
    want = torch.log_softmax(x, dim=1).gather(1, ids[:, None])[:, 0]
    xid = (x.gather(1, ids[:, None])[:, 0] - x.amax(dim=1)).abs()
    tol = 4 * E * (xid + 8) + 2.0 ** -21 + (vocab / 2048 + 64) * E + E * want.abs()
    got = logp.cpu().double()
    beyond = want < -MOST * (1 + E)                                  # rounds to infinity
    assert bool((got[beyond] == -math.inf).all()) and bool(((got - want).abs() <= tol)[~beyond].all())
    far = kind > 0                                                   # a ratio of 0: the bound's part of the loss, no gradient
    bound = weight * torch.where(adv < 0, -0.8 * adv, torch.zeros_like(adv))
    assert bool(((loss.cpu() - bound)[far].abs() <= 4 * E * bound[far]).all()) and bool((grad.cpu()[far] == 0).all())
