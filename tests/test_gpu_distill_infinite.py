"""A logit of +infinity makes the row's softmax NaN, wherever in the row it stands: also in the elements before and
after the vectors of 16 bytes, in rows that are held in registers and in those that are read twice."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_operators import distill_inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab,dtype", [(1001, "f32"), (40003, "f32"), (150001, "f32"), (1003, "bf16"), (262147, "bf16")])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_everywhere_in_the_row(pc, vocab, dtype, value):  # noqa: F811
    z, ids, t, w = distill_inputs(9, vocab, 7, dtype, masked=False)
    places = [0, 1, 2, vocab // 2, vocab - 1, vocab - 2, vocab - 3, None, None]
    for row, at in enumerate(places):
        if at is not None:
            z[row, at] = value
    z[7, 0] = z[7, vocab - 1] = -math.inf
    loss, grad = torch.zeros(9, device="cuda"), torch.zeros_like(z, device="cuda")
    sr.precond_distill(pc.h, z.cuda(), ids.cuda(), t.cuda(), loss, weight=(w + 0.1).cuda(), dlogits=grad)
    wl, wg = P.distill(z, ids, t, w + 0.1, 1.0)
    assert bool(wg[:7].isnan().all()) and bool(wg[7:].isfinite().all())
    assert torch.equal(loss.cpu().isnan(), wl.isnan())
    assert torch.equal(grad.cpu().isnan(), wg.isnan())
