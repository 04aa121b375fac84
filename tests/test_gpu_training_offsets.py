"""Rows whose offsets pass 32 bits: the layer norm, its gradients and the policy loss on matrices with a wide pitch."""
import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
import training_plain as T

pytestmark = pytest.mark.gpu
E, E16 = 2.0 ** -24, 2.0 ** -8
PITCH, ROWS = 2 ** 29 + 64, 9                        # the last rows begin beyond 2^32 elements


@pytest.fixture(scope="module")
def pc():
    p = sr.Preconditioner(0)
    yield p
    p.close()


def wide(x, pitch=PITCH):
    """x on the device with its rows `pitch` elements apart."""
    rows, cols = x.shape
    buf = torch.empty((rows - 1) * pitch + cols, dtype=x.dtype, device="cuda")
    v = buf.as_strided((rows, cols), (pitch, 1))
    v.copy_(x)
    return v


@pytest.mark.parametrize("cols", [640, 1001])
def test_layer_norm(pc, cols):
    g = P.generator(cols)
    x, dy, w, b = P.randn(g, ROWS, cols).bfloat16(), P.randn(g, ROWS, cols).bfloat16(), 1 + 0.3 * P.randn(g, cols), P.randn(g, cols)
    dx_in, y = wide(x), wide(torch.zeros_like(x))
    mean, rstd = torch.empty(ROWS, device="cuda"), torch.empty(ROWS, device="cuda")
    sr.precond_layer_norm(pc.h, dx_in, w.cuda(), 1e-5, bias=b.cuda(), y=y, mean=mean, rstd=rstd)
    _, want, m, r = T.layer_norm(x, None, w, b, 1e-5)
    # x is of order one: the mean within 64 E, rstd within 128 E of itself, y half a bf16 step more
    assert bool(((mean.cpu().double() - m).abs() <= 64 * E).all()) and bool(((rstd.cpu().double() - r).abs() <= 128 * E * r).all())
    assert bool(((y.cpu().double() - want).abs() <= E16 * want.abs() + 1e-4).all())
    del y
    out = wide(torch.zeros_like(x))
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    sr.precond_layer_norm_grad(pc.h, wide(dy), dx_in, w.cuda(), mean, rstd, out, dw, db=db)
    wx, ww, wb = T.layer_norm_grad(dy, x, w, mean.cpu(), rstd.cpu(), None)
    assert bool(((out.cpu().double() - wx).abs() <= E16 * wx.abs() + 1e-4).all())
    assert bool(((dw.cpu().double() - ww).abs() <= 1e-5).all()) and bool(((db.cpu().double() - wb).abs() <= 1e-5).all())


@pytest.mark.parametrize("vocab,in_place", [(2000, False), (5001, True)])
def test_policy(pc, vocab, in_place):
    g = P.generator(vocab)
    z = (2 * P.randn(g, ROWS, vocab)).bfloat16()
    ids, adv = torch.randint(0, vocab, (ROWS,), generator=g), P.randn(g, ROWS)
    dz = wide(z)
    grad = dz if in_place else wide(torch.zeros_like(z))
    loss, logp = torch.empty(ROWS, device="cuda"), torch.empty(ROWS, device="cuda")
    sr.precond_policy(pc.h, dz, ids.cuda(), advantage=adv.cuda(), loss=loss, logp=logp, dlogits=grad)
    wl, ws, wg = T.policy(z, ids, adv, None, None, None, 1.0, 0.2, 0.2, 0.0)
    assert bool(((logp.cpu().double() - ws).abs() <= 1e-5).all()) and bool(((loss.cpu().double() - wl).abs() <= 1e-5).all())
    assert bool(((grad.cpu().double() - wg).abs() <= E16 * wg.abs() + 1e-5 * adv.abs()[:, None]).all())
