"""A softmax does not change when all logits are shifted: the distillation loss and its gradient are as accurate for
logits around 1e5, or at a small temperature, as for those around 0.

Tolerance: E32 = 2^-24 is fp32's unit roundoff.  The exponent (z - max) / tau has a relative error of a few E32, so q one
of a few (spread / tau) E32, with spread the distance of the row's logits from their largest; sums and exponentials add
32 E32.  The offset does not come into it."""
import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_operators import E16, E32, distill_inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


def check(pc, z, ids, t, w, tau):  # noqa: F811
    rows, vocab = z.shape
    loss = torch.empty(rows, device="cuda")
    grad = torch.empty_like(z, device="cuda")
    sr.precond_distill(pc.h, z.cuda(), ids.cuda(), t.cuda(), loss, weight=w.cuda(), temperature=tau, dlogits=grad)
    wl, wg = P.distill(z, ids, t, w, tau)
    zd, td = z.double(), t.double()
    spread = ((zd.amax(dim=1) - zd.amin(dim=1)) + (td.amax(dim=1) - td.amin(dim=1))) / tau
    unit = (4 * spread + 32) * E32
    wt = w.double()
    assert bool(((loss.cpu().double() - wl).abs() <= wt * tau * tau * unit + 4 * E32 * wl.abs()).all())
    # the gradient: relative to q; where a candidate's q - p cancels, relative to their sum (at most 1 each)
    cand = torch.zeros(rows, vocab, dtype=torch.float64)
    cand.scatter_add_(1, ids.clamp(min=0).long(), (ids >= 0).double())
    tol = 3 * unit[:, None] * (wg.abs() + cand.clamp(max=1) * (wt * tau)[:, None]) + 1e-30
    if z.dtype == torch.bfloat16:
        tol = tol + E16 * wg.abs()
    bad = (grad.cpu().double() - wg).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((grad.cpu().double() - wg).abs() / tol).max()))


SIZES = [
    (6, 1000, 16),          # one block a row
    (8, 32000, 20),         # a cluster
    (400, 999, 5),
    (1900, 1500, 20),       # candidates in a kernel of their own
    (3, 150001, 30),        # rows that are read twice (fp32)
]


@pytest.mark.parametrize("offset", [1e3, 1e5, -6e5, 1e6])
@pytest.mark.parametrize("rows,vocab,top", SIZES)
def test_offset(pc, rows, vocab, top, offset):  # noqa: F811
    z, ids, t, w = distill_inputs(rows, vocab, top, "f32")
    check(pc, z + offset, ids, t + offset / 7, w, 1.0)


@pytest.mark.parametrize("rows,vocab,top", SIZES)
def test_small_temperature(pc, rows, vocab, top):  # noqa: F811
    z, ids, t, w = distill_inputs(rows, vocab, top, "f32")
    check(pc, z / 100 + 40, ids, t / 100, w, 0.01)


def test_offset_bf16(pc):  # noqa: F811
    """bf16 logits around 1000 lie 4 or 8 apart; rows that are read twice, too."""
    for rows, vocab, top in ((8, 32000, 20), (2, 263001, 9)):
        z, ids, t, w = distill_inputs(rows, vocab, top, "f32")
        check(pc, (4 * z + 1000).bfloat16(), ids, t, w, 2.0)


@pytest.mark.parametrize("rows,vocab,top", [(9, 40000, 20), (2, 150001, 9)])
def test_parts_of_very_different_size(pc, rows, vocab, top):  # noqa: F811
    """Lanes whose largest logits lie on both sides of the change of form (|max| / tau near 10^6 / log2(e))."""
    z, ids, t, w = distill_inputs(rows, vocab, top, "f32", masked=False)
    z = z + torch.where(torch.arange(vocab) % 64 < 40, 693145.0, 693150.0)
    check(pc, z, ids, t, w, 1.0)
    z[:, ::3] = -1e7
    z[:, 5::11] = 0
    ids = torch.arange(1, 3 * top, 3, dtype=torch.int32)[None].expand(rows, top).contiguous()
    assert bool((z.gather(1, ids.long()) != -1e7).all())
    check(pc, z, ids, t, w, 1.0)
