"""Matrices that are column slices of one buffer share no element though their spans do: outputs may lie beside inputs
there.  Slices that do share elements, or whose rows are not equally far apart, are refused."""
import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_operators_refusals import BASE, distill, gemm, grad, h, norm, quantize  # noqa: F401  (h: a host-only handle)

A = BASE["a"]
X = dict(rows=4, cols=256, ldx=1024, ldr=1024, ldt=1024, ldy=1024)          # bf16 slices of rows of 1024


@pytest.mark.parametrize("f,kw", [
    (norm, dict(X, x=A, r=A + 512, total=A + 1024, y=A + 1536)),
    (norm, dict(X, x=A, r=A + 512, total=A, y=A + 1536)),                    # total over x, beside the others
    (norm, dict(X, x=A + 1536, r=A + 1024, total=A + 512, y=A)),             # outputs before the inputs
    (norm, dict(X, x=A, y=A + 512 - 2048 * 2)),                              # rows of the one begin two rows earlier
    (norm, dict(X, x=A, y=A + 512 + 2048 * 3)),                              # and three later
    (grad, dict(lddy=1024, ldx=1024, lddr=1024, lddx=1024, dy=A, x=A + 512, dr=A + 1024, dx=A + 1536)),
    (quantize, dict(dtype=2, xs=BASE["f"], x=A, ldx=512, q=A + 208, ldq=512)),
    (gemm, dict(a=A, lda=96, b=A + 32, ldb=96, c=A + 64, n=8, dtype=0, ldc=24)),
    (distill, dict(z=A, ldz=2000, dz=A + 2000, lddz=2000))])
def test_accepts_slices(h, f, kw):  # noqa: F811
    assert f({**dict(h=h), **kw}) == sr.ENODEV


@pytest.mark.parametrize("f,kw", [
    (norm, dict(X, x=A, r=A + 512, total=A + 1022, y=A + 1536)),             # one element of the residual
    (norm, dict(X, x=A, y=A + 510)),
    (norm, dict(X, x=A, y=A + 1538)),                                        # its last element is x's next row's first
    (norm, dict(X, x=A + 2, y=A + 1540 - 2048 * 2)),
    (norm, dict(X, x=A, y=A + 512, ldy=1016)),                               # not equally far apart
    (grad, dict(lddy=1024, ldx=1024, lddr=1024, lddx=1024, dy=A, x=A + 512, dr=A + 1024, dx=A + 1026)),
    (quantize, dict(dtype=2, xs=BASE["f"], x=A, ldx=512, q=A + 192, ldq=512)),
    (gemm, dict(a=A, lda=96, b=A + 32, ldb=96, c=A + 60, n=8, dtype=0, ldc=24)),
    (distill, dict(z=A, ldz=2000, dz=A + 1998, lddz=2000))])
def test_refuses_what_shares_elements(h, f, kw):  # noqa: F811
    assert f({**dict(h=h), **kw}) == sr.EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols,gap", [(256, 0), (1000, 0), (1001, 3), (333, 1), (9000, 1)])
def test_slices_give_what_tensors_give(cols, gap, dtype):
    pc = sr.Preconditioner(0)
    g = P.generator(cols)
    rows, wide = 300, cols + gap
    buf = torch.full((rows, 5 * wide + gap), 7.0).to(dtype).cuda()
    x, r, total, y, dx = (buf[:, gap + i * wide:gap + i * wide + cols] for i in range(5))
    a, b, w = P.randn(g, rows, cols).to(dtype).cuda(), P.randn(g, rows, cols).to(dtype).cuda(), P.randn(g, cols).cuda()
    want_t, want_y, want_dx = (torch.empty(rows, cols, dtype=dtype, device="cuda") for _ in range(3))
    rstd, dw, dw2 = (torch.empty(n, device="cuda") for n in (rows, cols, cols))
    x.copy_(a)
    r.copy_(b)
    sr.precond_rms_norm(pc.h, a, w, 1e-6, residual=b, total=want_t, y=want_y, rstd=rstd)
    sr.precond_rms_norm_grad(pc.h, a, want_t, w, rstd, want_dx, dw, dresidual=b)
    sr.precond_rms_norm(pc.h, x, w, 1e-6, residual=r, total=total, y=y)
    sr.precond_rms_norm_grad(pc.h, x, total, w, rstd, dx, dw2, dresidual=r)
    # sums go in another order where rows do not begin at sectors: a few units of the last place, as the norm's own tests
    near = lambda p, q: bool(((p.double() - q.double()).abs() <= (cols / 16 + 48) * 2.0 ** -24 * (1 + q.double().abs().amax())
                              + (2.0 ** -8 * q.double().abs() if dtype == torch.bfloat16 else 0)).all())
    assert torch.equal(total, want_t) and torch.equal(x, a) and torch.equal(r, b)
    assert near(y, want_y) and near(dx, want_dx)
    for i in range(6):
        if gap:
            assert bool((buf[:, i * wide:i * wide + gap] == 7.0).all())
    pc.close()
