"""The policy loss of taken tokens that the logits forbid, in every kernel: rows in a warp's registers, in a warp's shared
memory, few rows, several blocks a row, rows that are read twice."""
import math

import pytest
import torch

import shampoo_roots_gb300 as sr
from test_gpu_policy import E, HIGH, LOW, inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu
SHAPES = [(40, 700, "bf16"), (200, 3001, "bf16"), (9, 40001, "bf16"), (200, 50001, "f32"), (4, 500003, "f32")]


def call(pc, z, ids, adv, old, ref, weight, tau, kl):  # noqa: F811
    rows = z.shape[0]
    loss, logp, grad = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(z, device="cuda")
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=old.cuda(), ref_logp=ref.cuda() if kl else None,
                      weight=weight.cuda(), temperature=tau, clip_low=LOW, clip_high=HIGH, kl=kl, loss=loss, logp=logp, dlogits=grad)
    return loss.cpu(), logp.cpu(), grad.cpu()


@pytest.mark.parametrize("rows,vocab,dtype", SHAPES)
def test_no_probability(pc, rows, vocab, dtype):  # noqa: F811
    """A logit of -infinity: logp -infinity; the loss is finite without the KL term (ratio 0) and infinite with it."""
    z, ids, adv, old, ref, weight = inputs(rows, vocab, dtype, 1.0)
    z[:, ::7] = -math.inf
    forbidden = torch.arange(rows) % 3 == 1
    ids = torch.where(forbidden, ids // 7 * 7, torch.where(ids % 7 == 0, ids + 1, ids)).clamp(max=vocab - 1)
    ids = torch.where(~forbidden & (ids % 7 == 0), ids - 1, ids)
    assert bool((torch.isneginf(z.gather(1, ids[:, None])[:, 0]) == forbidden).all())
    for kl in (0.0, 0.05):
        loss, logp, grad = call(pc, z, ids, adv, old, ref, weight, 1.0, kl)
        assert bool((logp[forbidden] == -math.inf).all())
        if kl:
            assert bool((loss[forbidden] == math.inf).all())
        else:                                                        # min(0 A, (1 - low) A): nothing of the token, or the bound's
            want = (weight * torch.where(adv < 0, -(1 - LOW) * adv, torch.zeros_like(adv)))[forbidden]
            assert bool(((loss[forbidden] - want).abs() <= 4 * E * want).all()) and bool((grad[forbidden] == 0).all())
        # the other rows are those of a call that leaves the forbidden ones out
        l2, s2, g2 = call(pc, z, ids, adv, old, ref, torch.where(forbidden, torch.zeros(()), weight), 1.0, kl)
        assert torch.equal(loss[~forbidden], l2[~forbidden]) and torch.equal(logp[~forbidden], s2[~forbidden])
        assert torch.equal(grad[~forbidden], g2[~forbidden]) and bool(torch.isfinite(g2).all())
