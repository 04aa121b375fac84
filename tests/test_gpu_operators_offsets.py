"""Offsets that pass 32 bits: rows 2^29 elements apart, so that the last of nine begins beyond 2^32 elements, give what
dense rows give."""
import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_operators import bytes_of, distill_inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu
ROWS, PITCH = 9, 1 << 29


@pytest.fixture(scope="module")
def wide():
    """Nine rows of 2^29 bf16 elements (9.7 GB); the matrices are column slices of it."""
    buf = torch.zeros(ROWS, PITCH, dtype=torch.bfloat16, device="cuda")
    yield buf
    del buf
    torch.cuda.empty_cache()


def slices(wide, cols, n, dtype=torch.bfloat16):
    b = wide.view(dtype)
    return [b[:, 4096 * i + 4096:4096 * i + 4096 + cols] for i in range(n)]


@pytest.mark.parametrize("cols", [640, 1001])
def test_norm_and_gradients(pc, wide, cols):  # noqa: F811
    g = P.generator(cols)
    a, b = (P.randn(g, ROWS, cols).bfloat16().cuda() for _ in range(2))
    w = P.randn(g, cols).cuda()
    x, r, t, y, dx = slices(wide, cols, 5)
    q8 = wide.view(torch.float8_e4m3fn)[:, 1 << 20:(1 << 20) + cols]
    x.copy_(a)
    r.copy_(b)
    q, s = sr.empty8(ROWS, cols)
    s2 = torch.empty_like(s)
    t1, y1, dx1 = (torch.empty_like(a) for _ in range(3))
    rs, rs2, dw, dw2 = (torch.empty(n, device="cuda") for n in (ROWS, ROWS, cols, cols))
    sr.precond_rms_norm(pc.h, a, w, 1e-6, residual=b, total=t1, y=y1, q=q, scale=s, rstd=rs)
    sr.precond_rms_norm(pc.h, x, w, 1e-6, residual=r, total=t, y=y, q=q8, scale=s2, rstd=rs2)
    assert torch.equal(t, t1) and torch.equal(bytes_of(s), bytes_of(s2))
    near = (cols / 32 + 16) * 2.0 ** -24               # the sums' order may differ: rows at other alignments
    assert bool(((rs2 - rs).abs() <= 2 * near * rs).all())
    assert bool(((y.float() - y1.float()).abs() <= (2.0 ** -7 + 2 * near) * y1.float().abs()).all())
    assert bool(((q8.float() - q.float()).abs() <= 2.0 ** -3 * q.float().abs() + 2.0 ** -9).all())
    sr.precond_rms_norm_grad(pc.h, b, t1, w, rs, dx1, dw, dresidual=a)
    sr.precond_rms_norm_grad(pc.h, r, t, w, rs, dx, dw2, dresidual=x)
    size = float(dx1.abs().max())
    assert bool(((dx.float() - dx1.float()).abs() <= 2.0 ** -7 * dx1.float().abs() + 2 * near * size).all())
    assert bool(((dw2 - dw).abs() <= 2 * near * (1 + dw.abs().max())).all())


@pytest.mark.parametrize("cols", [640, 1001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize(pc, wide, cols, dtype):  # noqa: F811
    a = P.randn(P.generator(cols), ROWS, cols).to(dtype).cuda()
    x = wide.view(dtype)[:, 4096:4096 + cols]
    q8 = wide.view(torch.float8_e4m3fn)[:, 1 << 20:(1 << 20) + cols]
    x.copy_(a)
    (q, s), (qt, st), (qt2, st2) = sr.empty8(ROWS, cols), sr.empty8(cols, ROWS), sr.empty8(cols, ROWS)
    s2 = torch.empty_like(s)
    sr.precond_quantize8(pc.h, a, q=q, scale=s, qt=qt, scale_t=st)
    sr.precond_quantize8(pc.h, x, q=q8, scale=s2, qt=qt2, scale_t=st2)
    assert torch.equal(bytes_of(q8), bytes_of(q)) and torch.equal(bytes_of(qt), bytes_of(qt2))
    assert torch.equal(bytes_of(s), bytes_of(s2)) and torch.equal(bytes_of(st), bytes_of(st2))
    # a matrix in 8-bit form, and transposed into rows far apart
    sr.precond_quantize8(pc.h, q8, x_scale=s2, qt=qt2, scale_t=st2)
    sr.precond_quantize8(pc.h, q, x_scale=s, qt=qt, scale_t=st)
    assert torch.equal(bytes_of(qt), bytes_of(qt2)) and torch.equal(bytes_of(st), bytes_of(st2))


@pytest.mark.parametrize("n", [128, 333])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_product(pc, wide, n, out):  # noqa: F811
    k = 1000
    g = P.generator(n)
    a, b = sr.empty8(ROWS, k), sr.empty8(n, k)
    sr.precond_quantize8(pc.h, P.randn(g, ROWS, k).cuda(), *a)
    sr.precond_quantize8(pc.h, P.randn(g, n, k).cuda(), *b)
    far = wide.view(torch.float8_e4m3fn)[:, 1 << 20:(1 << 20) + k]
    far.view(torch.uint8).copy_(a[0].view(torch.uint8))
    c = wide.view(out)[:, 4096:4096 + n]
    want = torch.empty(ROWS, n, dtype=out, device="cuda")
    sr.precond_gemm8(pc.h, *a, *b, want)
    sr.precond_gemm8(pc.h, far, a[1], *b, c)
    assert torch.equal(c, want)
    if out == torch.float32:
        sr.precond_gemm8(pc.h, far, a[1], *b, c, accumulate=True)
        assert torch.equal(c, 2 * want)
    sr.precond_gemm8_status(pc.h)


@pytest.mark.parametrize("vocab", [1001, 66001])
def test_distillation(pc, wide, vocab):  # noqa: F811
    z, ids, t, w = (v.cuda() for v in distill_inputs(ROWS, vocab, 9, "bf16"))
    far, dz = (wide[:, o:o + vocab] for o in (4096, 1 << 17))
    far.copy_(z)
    want, loss, loss2 = torch.empty_like(z), torch.empty(ROWS, device="cuda"), torch.empty(ROWS, device="cuda")
    sr.precond_distill(pc.h, z, ids, t, loss, weight=w, dlogits=want)
    sr.precond_distill(pc.h, far, ids, t, loss2, weight=w, dlogits=dz)
    near = lambda a, b, e: bool(((a.double() - b.double()).abs() <= e * b.double().abs() + 1e-5).all())
    assert near(loss2, loss, 1e-5) and near(dz, want, 2.0 ** -7)
