"""The training-step operators on the GPU against the plain 64-bit forms (tests/operators_plain.py).

Tolerances: eps32 = 2^-24 is fp32's unit roundoff.  A sum of n fp32 terms split over the threads of a row is within
(n / 32 + 16) eps32 of the sum of magnitudes; e4m3 rounds within 2^-4 of a value or 2^-10 of the scale; bf16 (8 significant bits) within
2^-8."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr

pytestmark = pytest.mark.gpu
E32, E16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def pc():
    p = sr.Preconditioner(0)
    yield p
    p.close()


def put8(x, tile=False, pitch=None):
    """A matrix in 8-bit form on the GPU, made by the plain form; and its float64 values."""
    q, e = P.quantize(x, tile)
    rows, cols = x.shape
    dq, ds = sr.empty8(rows, cols)
    if pitch:
        dq = torch.full((rows, pitch), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :cols]
    dq.copy_(q.to(torch.float32).to(torch.float8_e4m3fn))
    ds.view(torch.uint8).view(-1).copy_(P.order_scales(e, rows, cols))
    return dq, ds, P.dequantize(q, e)


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu()


def same8(q, s, want, exps, what):
    rows, cols = want.shape
    assert torch.equal(q.float().cpu().double().nan_to_num(nan=1e9), want.nan_to_num(nan=1e9)), what
    assert torch.equal(bytes_of(s).view(-1), P.order_scales(exps, rows, cols)), what + " scales"


# ------------------------------------------------------------------------------------------------ 8-bit form
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 128), (128, 128), (127, 129), (129, 640), (200, 1000), (31, 2049),
                                       (513, 72)])
def test_quantize(pc, rows, cols, tile, dtype):
    g = P.generator(rows * 10007 + cols)
    x = P.randn(g, rows, cols) * torch.exp(4 * P.randn(g, rows, 1))
    x[rows // 2, : cols // 2] = 0
    x = x.to(TYPES[dtype])
    dx = x.cuda()
    q, s = sr.empty8(rows, cols)
    qt, st = sr.empty8(cols, rows)
    sr.precond_quantize8(pc.h, dx, q=q, scale=s, qt=qt, scale_t=st, block=sr.BLOCK_TILE if tile else sr.BLOCK_ROW)
    want, e = P.quantize(x, tile)
    same8(q, s, want, e, "rows")
    want, e = P.quantize(x.t().contiguous(), tile)
    same8(qt, st, want, e, "columns")
    # each way alone gives the same
    q2, s2 = sr.empty8(rows, cols)
    qt2, st2 = sr.empty8(cols, rows)
    block = sr.BLOCK_TILE if tile else sr.BLOCK_ROW
    sr.precond_quantize8(pc.h, dx, q=q2, scale=s2, block=block)
    sr.precond_quantize8(pc.h, dx, qt=qt2, scale_t=st2, block=block)
    for a, b in ((q, q2), (s, s2), (qt, qt2), (st, st2)):
        assert torch.equal(bytes_of(a), bytes_of(b))


@pytest.mark.parametrize("tile", [False, True])
def test_quantize_values(pc, tile):
    """Zeros, subnormals, the largest numbers, boundaries of two scales, infinities and NaN."""
    x = torch.zeros(130, 300)
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = 1e-45, 1.2e-38, 3.4e38, -3.4e38
    for i, v in enumerate([448.0, math.nextafter(448.0, 1e9), 449.0, 464.0, 224.0, 224.00002, 2.0 ** -100 * 448, 0.875, 1.75]):
        x[10 + i, 130 + i] = v
        x[10 + i, 140] = -v / 7
    x[40, 5], x[40, 6] = math.inf, 3.0
    x[41, 5], x[41, 6] = -math.inf, 2e-3
    x[42, 200], x[42, 6] = math.nan, 1.0
    x[43, :] = math.nan
    x[129, 299] = 7.0
    q, s = sr.empty8(130, 300)
    qt, st = sr.empty8(300, 130)
    sr.precond_quantize8(pc.h, x.cuda(), q=q, scale=s, qt=qt, scale_t=st, block=sr.BLOCK_TILE if tile else sr.BLOCK_ROW)
    same8(q, s, *P.quantize(x, tile), "rows")
    same8(qt, st, *P.quantize(x.t().contiguous(), tile), "columns")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pitch,offset", [(1000, 0), (1003, 0), (1008, 1), (1008, 8)])
def test_quantize_pitch_and_alignment(pc, dtype, pitch, offset):
    x = P.randn(P.generator(5), 70, 1000).to(TYPES[dtype])
    dx = P.pitched(x, pitch, offset=offset)
    buf = torch.full((70, 1040), 0x55, dtype=torch.uint8, device="cuda")
    q = buf.view(torch.float8_e4m3fn)[:, :1000]
    s = sr.empty8(70, 1000)[1]
    sr.precond_quantize8(pc.h, dx, q=q, scale=s)
    same8(q, s, *P.quantize(x), "rows")
    assert bool((buf[:, 1000:] == 0x55).all())             # nothing is written between the rows


@pytest.mark.parametrize("rows,cols", [(1, 40), (130, 700), (300, 129)])
def test_quantize_of_8_bit_form(pc, rows, cols):
    """An activation in 8-bit form, put into blocks of tokens."""
    g = P.generator(rows)
    dq, ds, v = put8(P.randn(g, rows, cols) * torch.exp(2 * P.randn(g, rows, 1)))
    qt, st = sr.empty8(cols, rows)
    sr.precond_quantize8(pc.h, dq, x_scale=ds, qt=qt, scale_t=st)
    same8(qt, st, *P.quantize(v.float().t().contiguous()), "columns")
    q, s = sr.empty8(rows, cols)
    sr.precond_quantize8(pc.h, dq, x_scale=ds, q=q, scale=s)
    assert torch.equal(sr.dequantize8(q, s).cpu().double(), v)


# ------------------------------------------------------------------------------------------------ norm
def check_norm(pc, rows, cols, dtype, wtype, residual, seed=0, eps=1e-6, pitch=0, scale=1.0):
    g = P.generator(seed + rows * 31 + cols)
    x = (scale * P.randn(g, rows, cols) * torch.exp(P.randn(g, rows, 1))).to(TYPES[dtype])
    r = (scale * P.randn(g, rows, cols)).to(TYPES[dtype]) if residual else None
    w = (1 + 0.3 * P.randn(g, cols)).to(TYPES[wtype])
    place = (lambda t: P.pitched(t, cols + pitch, offset=pitch % 5)) if pitch else (lambda t: t.cuda())
    dx = place(x)
    dr = place(r) if residual else None
    total = torch.empty_like(x, device="cuda") if residual else None
    y = torch.empty_like(x, device="cuda")
    q, s = sr.empty8(rows, cols)
    rstd = torch.empty(rows, device="cuda")
    sr.precond_rms_norm(pc.h, dx, w.cuda(), eps, residual=dr, total=total, y=y, q=q, scale=s, rstd=rstd)
    h, want, rs = P.rms_norm(x, r, w, eps)
    if residual:
        assert torch.equal(total.cpu(), h)
    near = (cols / 32 + 16) * E32                           # of the mean square, half of it of rstd
    assert bool(((rstd.cpu().double() - rs).abs() <= (near + 4 * E32) * rs).all())
    out = y.cpu().double()
    assert bool(((out - want).abs() <= want.abs() * (near + 8 * E32 + (E16 if dtype == "bf16" else 0)) + 1e-38).all())
    # the 8-bit form: the scale fits the block, and each value is a nearest one
    sc = sr.scales8(s, rows, cols).cpu().double()
    v = torch.zeros(rows, P.blocks(cols) * 128, dtype=torch.float64)
    v[:, :cols] = want.abs()
    amax = v.view(rows, -1, 128).amax(dim=2)
    tol = 1 + 2 * near + 16 * E32
    empty = amax == 0
    assert bool(((amax <= 448 * sc * tol) & ((amax * tol > 224 * sc) | empty)).all())
    assert bool((sc[empty] == 1).all())
    got = sr.dequantize8(q, s).cpu().double()
    each = sc.repeat_interleave(128, dim=1)[:, :cols]
    assert bool(((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, each * 2.0 ** -10) * 1.001 + want.abs() * (tol - 1)).all())
    pad = P.order_scales(torch.zeros(rows, P.blocks(cols), dtype=torch.int64), rows, cols)
    assert bool((bytes_of(s).view(-1)[pad == 127] == 127).all())
    # outputs left out change nothing in the others
    q2, s2 = sr.empty8(rows, cols)
    t2 = torch.empty_like(total) if residual else None
    sr.precond_rms_norm(pc.h, dx, w.cuda(), eps, residual=dr, total=t2, q=q2, scale=s2)
    assert torch.equal(bytes_of(q), bytes_of(q2)) and torch.equal(bytes_of(s), bytes_of(s2))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (1, 1024), (3, 100), (5, 128), (130, 256), (257, 1000), (33, 4096),
                                       (17, 4104), (9, 6144), (7, 8200), (5, 16384), (3, 16392), (2, 40000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rms_norm(pc, rows, cols, dtype):
    check_norm(pc, rows, cols, dtype, "f32", True)
    check_norm(pc, rows, cols, dtype, "bf16", False)


@pytest.mark.parametrize("cols", [72, 1001, 5000, 20001])
def test_rms_norm_pitch(pc, cols):
    check_norm(pc, 19, cols, "bf16", "f32", True, pitch=3)
    check_norm(pc, 19, cols, "f32", "f32", True, pitch=8)


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(500, 48, "bf16", 0), (77, 130, "bf16", 14), (301, 256, "f32", 0), (40, 7001, "bf16", 0),
                                                   (90, 6146, "f32", 6), (77, 13001, "bf16", 1), (50, 24577, "f32", 0), (45, 49153, "bf16", 0),
                                                   (700, 1213, "bf16", 0), (330, 2009, "f32", 0), (200, 530, "bf16", 1)])
def test_rms_norm_layouts(pc, rows, cols, dtype, pitch):
    """Several rows in a warp, rows at every alignment, rows shared by 2, 4 and 8 blocks and longer ones; more rows than run at once."""
    check_norm(pc, rows, cols, dtype, "f32", True, pitch=pitch)
    check_norm(pc, rows, cols, dtype, "bf16", False, pitch=pitch)


def test_rms_norm_values(pc):
    """Rows of zeros, of tiny and of large numbers, a NaN row; its neighbours keep their values."""
    check_norm(pc, 64, 640, "f32", "f32", False, scale=1e-12)
    check_norm(pc, 64, 640, "f32", "f32", False, scale=1e15)
    x = P.randn(P.generator(1), 40, 512)
    x[3] = 0
    x[7, 100] = math.nan
    x[9, 5] = math.inf
    y = torch.empty(40, 512, device="cuda")
    q, s = sr.empty8(40, 512)
    sr.precond_rms_norm(pc.h, x.cuda(), torch.ones(512, device="cuda"), 1e-6, y=y, q=q, scale=s)
    _, want, _ = P.rms_norm(x, None, torch.ones(512), 1e-6)
    y, d = y.cpu().double(), sr.dequantize8(q, s).cpu().double()
    assert bool((y[3] == 0).all()) and bool((d[3] == 0).all())
    assert bool(y[7].isnan().all()) and bool(d[7].isnan().all())
    assert bool(y[9, 5].isnan()) and bool((y[9, :5] == 0).all()) and bool(d[9, 5].isnan())
    keep = torch.ones(40, dtype=torch.bool)
    keep[[3, 7, 9]] = False
    assert bool(((y - want)[keep].abs() <= want[keep].abs() * 40 * E32).all())
    assert bool(((d - want)[keep].abs() <= want[keep].abs() * 2.0 ** -4 * 1.001 + 2.0 ** -10 * 448).all())


@pytest.mark.parametrize("cols", [1000, 20000])
def test_rms_norm_in_place(pc, cols):
    g = P.generator(3)
    x, r = P.randn(g, 21, cols), P.randn(g, 21, cols)
    for over in ("x", "residual"):
        dx, dr = x.cuda(), r.cuda()
        y, y2 = torch.empty(21, cols, device="cuda"), torch.empty(21, cols, device="cuda")
        t = torch.empty(21, cols, device="cuda")
        sr.precond_rms_norm(pc.h, dx, torch.ones(cols, device="cuda"), 1e-6, residual=dr, total=t, y=y)
        sr.precond_rms_norm(pc.h, dx, torch.ones(cols, device="cuda"), 1e-6, residual=dr, total=dx if over == "x" else dr, y=y2)
        assert torch.equal(t, dx if over == "x" else dr) and torch.equal(y, y2)


def check_grad(pc, rows, cols, dtype, residual, pitch=0):
    g = P.generator(rows * 77 + cols)
    x = P.randn(g, rows, cols).to(TYPES[dtype])
    dy = (P.randn(g, rows, cols) * torch.exp(2 * P.randn(g, rows, 1))).to(TYPES[dtype])
    dr = P.randn(g, rows, cols).to(TYPES[dtype]) if residual else None
    w = 1 + 0.3 * P.randn(g, cols)
    rstd = P.rms_norm(x, None, w, 1e-6)[2].float()
    place = (lambda t: P.pitched(t, cols + pitch, offset=pitch % 5)) if pitch else (lambda t: t.cuda())
    dx = torch.full((rows, cols), math.nan, device="cuda").to(TYPES[dtype])
    dw = torch.full((cols,), math.nan, device="cuda")
    d_dr = place(dr) if residual else None
    sr.precond_rms_norm_grad(pc.h, place(dy), place(x), w.cuda(), rstd.cuda(), dx, dw, dresidual=d_dr)
    wx, ww = P.rms_norm_grad(dy, x, w, rstd, dr)
    f = lambda t: t.double()
    n = (f(x) * f(rstd)[:, None]).abs()
    gw = (f(dy) * f(w)).abs()
    size = f(rstd)[:, None] * (gw + n * (gw * n).mean(dim=1, keepdim=True)) + (f(dr).abs() if residual else 0)
    tol = (cols / 32 + 24) * E32 * size + (E16 * wx.abs() if dtype == "bf16" else 0) + 1e-38
    assert bool(((dx.cpu().double() - wx).abs() <= tol).all())
    assert bool(((dw.cpu().double() - ww).abs() <= (rows / 8 + 48) * E32 * (f(dy).abs() * n).sum(dim=0) + 1e-38).all())
    return dict(x=x, dy=dy, dr=dr, w=w, rstd=rstd, dx=dx, dw=dw)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (2, 1024), (300, 100), (1000, 256), (77, 1000), (40, 4096), (33, 4104),
                                       (9, 8192), (7, 8200), (5, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rms_norm_grad(pc, rows, cols, dtype):
    check_grad(pc, rows, cols, dtype, True)
    check_grad(pc, rows, cols, dtype, False)


def test_rms_norm_grad_pitch(pc):
    check_grad(pc, 19, 1001, "bf16", True, pitch=3)
    check_grad(pc, 19, 1000, "f32", True, pitch=8)
    check_grad(pc, 5, 9001, "bf16", True, pitch=3)


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(3000, 48, "bf16", 0), (77, 130, "bf16", 14), (1001, 256, "f32", 0), (200, 9001, "bf16", 0),
                                                   (190, 6146, "f32", 6), (77, 17000, "bf16", 8), (50, 24577, "f32", 0), (45, 49153, "bf16", 1),
                                                   (2000, 1213, "bf16", 0), (600, 2009, "f32", 0), (900, 530, "bf16", 1)])
def test_rms_norm_grad_layouts(pc, rows, cols, dtype, pitch):
    check_grad(pc, rows, cols, dtype, True, pitch=pitch)
    check_grad(pc, rows, cols, dtype, False, pitch=pitch)


def test_rms_norm_grad_in_place(pc):
    c = check_grad(pc, 50, 640, "bf16", True)
    for over in ("dy", "dr", "x"):
        d = {k: c[k].cuda() for k in ("x", "dy", "dr", "w", "rstd")}
        dw = torch.empty(640, device="cuda")
        sr.precond_rms_norm_grad(pc.h, d["dy"], d["x"], d["w"], d["rstd"], d[over], dw, dresidual=d["dr"])
        assert torch.equal(d[over], c["dx"]) and torch.equal(dw, c["dw"])


def test_rms_norm_grad_against_differences(pc):
    """<dx, u> and <dw, v> against central differences of the 64-bit norm along random directions."""
    g = P.generator(12)
    rows, cols, eps = 6, 300, 1e-3
    x, dy, w = P.randn(g, rows, cols), P.randn(g, rows, cols), 1 + 0.3 * P.randn(g, cols)
    rstd = torch.empty(rows, device="cuda")
    sr.precond_rms_norm(pc.h, x.cuda(), w.cuda(), eps, rstd=rstd)
    dx, dw = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
    sr.precond_rms_norm_grad(pc.h, dy.cuda(), x.cuda(), w.cuda(), rstd, dx, dw)
    f = lambda a, b: float((P.rms_norm(a, None, b, eps)[1] * dy.double()).sum())
    x, w, step = x.double(), w.double(), 1e-5
    for _ in range(4):
        u, v = P.randn(g, rows, cols).double(), P.randn(g, cols).double()
        along_x = (f(x + step * u, w) - f(x - step * u, w)) / (2 * step)
        along_w = (f(x, w + step * v) - f(x, w - step * v)) / (2 * step)
        # differences of an fp64 sum of about 50: step^2 and 1e-16 * 50 / step, both below 1e-7
        assert abs(float((dx.cpu().double() * u).sum()) - along_x) <= 1e-4
        assert abs(float((dw.cpu().double() * v).sum()) - along_w) <= 1e-4


# ------------------------------------------------------------------------------------------------ product
def check_gemm(pc, m, n, k, out="bf16", accumulate=False, tile=True, seed=0, pitch=0, ldc=0):
    g = P.generator(seed + m * 131 + n * 17 + k)
    A = P.randn(g, m, k) * torch.exp(2 * P.randn(g, m, 1)) if k else torch.zeros(m, 0)
    B = P.randn(g, n, k) * torch.exp(P.randn(g, n, 1)) if k else torch.zeros(n, 0)
    rnd = -(-max(k, 1) // 16) * 16
    qa, sa, a = put8(A, pitch=rnd + 16 * pitch if pitch else None)
    qb, sb, b = put8(B, tile, pitch=rnd + 32 * pitch if pitch else None)
    c0 = P.randn(g, m, n)
    C = torch.full((m, ldc or n), 7.0, device="cuda").to(TYPES[out])
    c = C[:, :n]
    if accumulate:
        c.copy_(c0)
    sr.precond_gemm8(pc.h, qa, sa, qb, sb, c, accumulate=accumulate)
    sr.precond_gemm8_status(pc.h)
    want = a @ b.t() + (c0.double() if accumulate else 0)
    size = a.abs() @ b.abs().t() + (c0.double().abs() if accumulate else 0)
    # every 32 products round once, downwards (2^-23 of the sums' size at most); fp32 results also add a segment
    # every 512 columns
    chain = k / 32 + 8 if out == "bf16" else 24 + k / 512
    tol = chain * 2.0 ** -23 * size + (E16 * want.abs() if out == "bf16" else 0) + 1e-38
    bad = (c.cpu().double() - want).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())
    if ldc:
        assert bool((C[:, n:] == 7.0).all())
    return qa, sa, qb, sb, c


@pytest.mark.parametrize("m,n,k", [(128, 128, 128), (128, 128, 1024), (256, 384, 640), (1, 1, 1), (1, 128, 16), (1, 1000, 2000),
                                   (5, 333, 129), (16, 4096, 512), (17, 500, 3000), (33, 200, 1111), (64, 256, 4096), (65, 300, 700),
                                   (127, 129, 4100), (300, 20, 900), (500, 64, 100), (700, 5, 6000), (1000, 1000, 130), (129, 2000, 513),
                                   (2500, 1300, 256), (64, 64, 64), (40, 40, 5000)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm(pc, m, n, k, out):
    check_gemm(pc, m, n, k, out)


@pytest.mark.parametrize("m,n,k", [(1, 300, 700), (50, 129, 1000), (200, 140, 8191), (700, 33, 100), (1500, 1100, 1000)])
def test_gemm_accumulate(pc, m, n, k):
    check_gemm(pc, m, n, k, "f32", accumulate=True, tile=False)


@pytest.mark.parametrize("m,n,k,ldc", [(3, 130, 300, 131), (200, 130, 300, 133), (200, 129, 300, 136), (129, 256, 77, 264)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_pitch(pc, m, n, k, ldc, out):
    check_gemm(pc, m, n, k, out, pitch=1, ldc=ldc)


@pytest.mark.parametrize("m,n,k,ldc", [(70, 300, 1024, 304), (130, 260, 2048, 264), (128, 128, 4096, 128), (129, 250, 4000, 251),
                                       (8, 128, 1024, 128), (20, 500, 2048, 512), (60, 300, 4096, 301), (16, 16, 3000, 16)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_stretches(pc, m, n, k, ldc, out):
    """Tiles that 2, 4 or 8 blocks share, a stretch of K each: results of 4 elements at a time and single ones."""
    check_gemm(pc, m, n, k, out, ldc=ldc)
    if out == "f32":
        check_gemm(pc, m, n, k, out, accumulate=True, ldc=ldc)


@pytest.mark.parametrize("m,n,k", [(0, 5, 5), (5, 0, 5), (130, 70, 0), (3, 200, 0)])
def test_gemm_empty(pc, m, n, k):
    check_gemm(pc, m, n, k, "f32")
    check_gemm(pc, m, n, k, "f32", accumulate=True)


def test_gemm_repeats(pc):
    """The same bits again, and from another stream."""
    for m, n, k in ((7, 900, 5000), (700, 900, 3000)):
        for out in ("bf16", "f32"):
            qa, sa, qb, sb, c = check_gemm(pc, m, n, k, out)
            other = torch.cuda.Stream()
            d = torch.empty_like(c)
            torch.cuda.synchronize()
            with torch.cuda.stream(other):
                for _ in range(3):
                    sr.precond_gemm8(pc.h, qa, sa, qb, sb, d)
            other.synchronize()
            assert torch.equal(c, d)


def test_gemm_small_sums_of_a_long_chain(pc):
    """A long chain of positive products, where truncated sums would drift: fp32 results stay within a segment's error."""
    k = 16384
    qa, sa, a = put8(torch.rand(130, k, generator=P.generator(1)) + 0.5)
    qb, sb, b = put8(torch.rand(140, k, generator=P.generator(2)) + 0.5)
    c = torch.empty(130, 140, device="cuda")
    sr.precond_gemm8(pc.h, qa, sa, qb, sb, c)
    want = a @ b.t()
    assert float(((c.cpu().double() - want) / want).abs().max()) <= (16 + 32) * 2.0 ** -24


# ------------------------------------------------------------------------------------------------ distillation
def distill_inputs(rows, vocab, top, dtype, seed=0, ids64=False, tdtype="f32", masked=True):
    g = P.generator(seed + rows * 7 + vocab)
    z = (3 * P.randn(g, rows, vocab)).to(TYPES[dtype])
    ids = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(rows)])
    t = (3 * P.randn(g, rows, top)).to(TYPES[tdtype])
    if masked:
        ids[torch.rand(rows, top, generator=g) < 0.2] = -1
    w = torch.rand(rows, generator=g)
    if masked:
        w[::4] = 0
    return z, ids if ids64 else ids.int(), t, w


def check_distill(pc, z, ids, t, w, tau, grad=True, place=None, in_place=False):
    place = place or (lambda x: x.cuda())
    dz = place(z)
    rows, vocab = z.shape
    loss = torch.full((rows,), math.nan, device="cuda")
    g = None
    if grad:
        g = dz if in_place else place(torch.full(z.shape, math.nan).to(z.dtype))
    sr.precond_distill(pc.h, dz, ids.cuda(), t.cuda(), loss, weight=None if w is None else w.cuda(), temperature=tau, dlogits=g)
    wl, wg = P.distill(z, ids, t, w, tau)
    wt = torch.ones(rows, dtype=torch.float64) if w is None else w.double()
    zmax = torch.where(z.double().isfinite(), z.double(), torch.zeros(1, dtype=torch.float64)).abs().amax(dim=1) / tau
    tmax = torch.where(t.double().isfinite(), t.double(), torch.zeros(1, dtype=torch.float64)).abs().amax(dim=1) / tau
    # a log-probability is a difference of numbers up to 2 max |logit| / tau, its exponentials a few ulp
    unit = (4 * (zmax + tmax) + 32) * E32
    fine = wl.isfinite()
    got = loss.cpu().double()
    assert torch.equal(got[~fine & ~wl.isnan()], wl[~fine & ~wl.isnan()]) and torch.equal(got.isnan(), wl.isnan())
    assert bool(((got - wl)[fine].abs() <= (wt * tau * tau * (unit + 1e-30))[fine] + 4 * E32 * wl[fine].abs()).all())
    if not grad:
        return loss, g
    got = g.cpu().double()
    assert torch.equal(got.isnan(), wg.isnan())
    got, want = got.nan_to_num(), wg.nan_to_num()
    # q's relative error is its logarithm's: |z - max| / tau and a few ulp; p likewise
    tol = (wt * tau)[:, None] * 3 * unit[:, None] * (want.abs() / (wt * tau)[:, None].clamp(min=1e-30) + 0) + 1e-30
    cand = torch.zeros(rows, vocab, dtype=torch.float64)
    ok = (ids >= 0) & (ids < vocab)
    cand.scatter_add_(1, ids.clamp(0, vocab - 1).long(), ok.double())
    cand = cand.clamp(max=1)
    tol = tol + cand * (wt * tau)[:, None] * 3 * unit[:, None]          # q - p of a candidate may cancel
    if z.dtype == torch.bfloat16:
        tol = tol + E16 * want.abs()
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist())
    return loss, g


@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 2, 2), (3, 7, 3), (9, 1000, 32), (5, 1001, 1), (40, 4096, 100), (2, 50001, 20),
                                            (4, 32768, 64), (1, 131072, 256), (7, 33333, 1000), (400, 999, 17), (330, 17000, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill(pc, rows, vocab, top, dtype):
    z, ids, t, w = distill_inputs(rows, vocab, top, dtype)
    check_distill(pc, z, ids, t, w, 2.0)
    check_distill(pc, z, ids, t, None, 0.7, grad=False)


@pytest.mark.parametrize("rows,vocab,top", [(700, 7, 3), (650, 333, 40), (1300, 1001, 5), (80, 70001, 300), (640, 2048, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_many_rows(pc, rows, vocab, top, dtype):
    """Rows whose candidates have a kernel of their own; some without candidates, some with one id throughout, in place."""
    top = min(top, vocab)
    z, ids, t, w = distill_inputs(rows, vocab, top, dtype)
    ids[5::9] = -1
    ids[7::11] = ids[7::11, :1]
    t[3::13] = -math.inf
    a = check_distill(pc, z, ids, t, w, 1.5)
    b = check_distill(pc, z, ids, t, w, 1.5, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = check_distill(pc, z, ids, t, w, 1.5, grad=False)
    assert torch.equal(a[0], c[0])


@pytest.mark.parametrize("rows,vocab,top", [(700, 1500, 129), (650, 3001, 256), (9, 5000, 200), (640, 400, 257)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_candidate_counts(pc, rows, vocab, top, dtype):
    z, ids, t, w = distill_inputs(rows, vocab, top, dtype)
    ids[1::3, 128:] = ids[1::3, :top - 128]                   # a second occurrence past the first 128
    check_distill(pc, z, ids, t, w, 1.5)


@pytest.mark.parametrize("rows,vocab,top", [(2000, 333, 40), (2100, 1001, 5), (1900, 3001, 200), (460, 70001, 30), (1900, 2048, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_very_many_rows(pc, rows, vocab, top, dtype):
    """As test_distill_many_rows, with more rows than run at once; every id twice in some."""
    z, ids, t, w = distill_inputs(rows, vocab, top, dtype)
    ids[5::9] = -1
    ids[7::11] = ids[7::11, :1]
    ids[2::17, top // 2:] = ids[2::17, :top - top // 2]
    t[3::13] = -math.inf
    a = check_distill(pc, z, ids, t, w, 1.5)
    b = check_distill(pc, z, ids, t, w, 1.5, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = check_distill(pc, z, ids, t, w, 1.5, grad=False)
    assert torch.equal(a[0], c[0])


def test_distill_types_and_places(pc):
    z, ids, t, w = distill_inputs(11, 1003, 24, "bf16", ids64=True, tdtype="bf16")
    check_distill(pc, z, ids, t, w, 1.0)
    for dtype in ("bf16", "f32"):
        z, ids, t, w = distill_inputs(11, 1003, 24, dtype)
        for pitch, offset in ((1003, 0), (1008, 0), (1011, 3)):
            check_distill(pc, z, ids, t, w, 1.0, place=lambda x: P.pitched(x, pitch, offset=offset))
        a = check_distill(pc, z, ids, t, w, 1.0)
        b = check_distill(pc, z, ids, t, w, 1.0, in_place=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        # logits and gradient of different alignment
        dz = z.cuda()
        g = P.pitched(torch.zeros_like(z), 1003, offset=1)
        loss = torch.empty(11, device="cuda")
        sr.precond_distill(pc.h, dz, ids.cuda(), t.cuda(), loss, weight=w.cuda(), dlogits=g)
        assert torch.equal(loss, a[0]) and torch.equal(g, a[1])


@pytest.mark.parametrize("vocab", [64, 40000])
def test_distill_masks(pc, vocab):
    """Rows without candidates, repeated ids, ids outside the vocabulary, masked logits, zero weights over NaN."""
    low = torch.finfo(torch.float32).min
    z, ids, t, w = distill_inputs(16, vocab, 12, "f32", masked=False)
    ids[0] = -1                                   # no candidate
    t[1] = -math.inf                              # none that the teacher gives anything
    ids[2] = ids[2, 0]                            # one id twelve times
    ids[3, 4:] = ids[3, :4].repeat(2)             # pairs
    ids[4, 0], ids[4, 1] = vocab, 2 ** 31 - 1     # outside
    z[5, vocab // 2:] = -math.inf
    ids[5] = torch.arange(12)
    z[6, 1:] = low                                # the type's lowest value
    ids[6] = torch.arange(12)
    t[6, 1:] = -math.inf
    z[7] = low
    z[8, 3:] = -math.inf
    ids[8] = torch.arange(12)
    t[8, 3:] = -math.inf                          # candidates of no weight at masked logits
    z[9] = math.nan
    w[9] = 0
    t[10, 1:] = low
    z[11] = 1e30                                  # large and equal
    ids[12, :11] = -1                             # one candidate: p = 1
    z[13] = z[13] * 1e-30
    w[14], w[15] = 1e-20, 1e20
    check_distill(pc, z, ids, t, w, 1.0)
    check_distill(pc, z, ids, t, w, 0.25)


def test_distill_masks_many_rows(pc):
    """The same kinds of rows, a hundred times each."""
    low = torch.finfo(torch.float32).min
    z, ids, t, w = distill_inputs(1100, 120, 12, "f32", masked=False)
    ids[0::11] = -1
    t[1::11] = -math.inf
    ids[2::11] = ids[2::11, :1]
    ids[3::11, 0], ids[3::11, 1] = 120, 2 ** 31 - 1
    z[4::11, 60:] = -math.inf
    ids[4::11] = torch.arange(12, dtype=torch.int32)
    z[5::11] = low
    z[6::11] = math.nan
    w[6::11] = 0
    z[7::11] = 1e30
    z[8::11, 1:] = low
    ids[8::11] = torch.arange(12, dtype=torch.int32)
    t[8::11, 1:] = -math.inf
    check_distill(pc, z, ids, t, w, 1.0)
    check_distill(pc, z, ids, t, w, 0.25, in_place=True)


def test_distill_unlikely_candidate(pc):
    """A candidate at -infinity: an infinite loss and a finite gradient.  A row of -infinity: NaN."""
    z, ids, t, w = distill_inputs(3, 500, 6, "f32", masked=False)
    z[0, ids[0, 2].long()] = -math.inf
    z[1] = -math.inf
    loss, g = torch.empty(3, device="cuda"), torch.empty(3, 500, device="cuda")
    sr.precond_distill(pc.h, z.cuda(), ids.cuda(), t.cuda(), loss, dlogits=g)
    assert float(loss[0]) == math.inf and bool(g[0].isfinite().all())
    p = torch.softmax(t[0].double(), 0)
    assert abs(float(g[0, ids[0, 2].long()]) + float(p[2])) <= 1e-6
    assert bool(loss[1].isnan()) and bool(g[1].isnan().all())
    assert bool(loss[2].isfinite()) and bool(g[2].isfinite().all())


def test_distill_against_differences(pc):
    g = P.generator(4)
    z, ids, t, w = distill_inputs(5, 200, 9, "f32")
    w = w + 0.1
    tau, step = 1.7, 1e-5
    loss, dz = torch.empty(5, device="cuda"), torch.empty(5, 200, device="cuda")
    sr.precond_distill(pc.h, z.cuda(), ids.cuda(), t.cuda(), loss, weight=w.cuda(), temperature=tau, dlogits=dz)
    for _ in range(4):
        u = P.randn(g, 5, 200).double()
        f = lambda s: float(P.distill(z.double() + s * u, ids, t, w, tau)[0].sum())
        assert abs(float((dz.cpu().double() * u).sum()) - (f(step) - f(-step)) / (2 * step)) <= 1e-4


# ------------------------------------------------------------------------------------------------ together
def test_streams_and_graphs(pc):
    """Every operator on a stream of its own and inside a CUDA graph gives what it gives on the current stream."""
    g = P.generator(8)
    rows, cols, vocab, top = 200, 700, 900, 11
    x = P.randn(g, rows, cols).bfloat16().cuda()
    r = P.randn(g, rows, cols).bfloat16().cuda()
    w = P.randn(g, cols).cuda()
    z, ids, t, wt = (a.cuda() for a in distill_inputs(rows, vocab, top, "bf16"))

    def outputs():
        e = torch.empty
        return dict(h=e(rows, cols, dtype=torch.bfloat16, device="cuda"), q=sr.empty8(rows, cols), rstd=e(rows, device="cuda"),
                    qt=sr.empty8(cols, rows), c=e(rows, rows, device="cuda"), loss=e(rows, device="cuda"),
                    dz=e(rows, vocab, dtype=torch.bfloat16, device="cuda"), dx=e(rows, cols, dtype=torch.bfloat16, device="cuda"),
                    dw=e(cols, device="cuda"), ws=e(sr.precond_rms_norm_grad_workspace(rows, cols), dtype=torch.uint8, device="cuda"))

    def go(o, stream=None):
        sr.precond_rms_norm(pc.h, x, w, 1e-6, residual=r, total=o["h"], q=o["q"][0], scale=o["q"][1], rstd=o["rstd"], stream=stream)
        sr.precond_quantize8(pc.h, x, qt=o["qt"][0], scale_t=o["qt"][1], stream=stream)
        sr.precond_gemm8(pc.h, *o["q"], *o["q"], o["c"], stream=stream)
        sr.precond_distill(pc.h, z, ids, t, o["loss"], weight=wt, dlogits=o["dz"], stream=stream)
        sr.precond_rms_norm_grad(pc.h, r, o["h"], w, o["rstd"], o["dx"], o["dw"], workspace=o["ws"], stream=stream)

    def flat(o):
        return [bytes_of(v) for k in ("h", "rstd", "c", "loss", "dz", "dx", "dw") for v in [o[k]]] + [bytes_of(v) for v in o["q"] + o["qt"]]

    first = outputs()
    go(first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    second = outputs()
    torch.cuda.synchronize()
    go(second, side)
    side.synchronize()
    third = outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(third)
    graph.replay()
    torch.cuda.synchronize()
    for o in (second, third):
        assert all(torch.equal(a, b) for a, b in zip(flat(first), flat(o)))


def test_empty_calls(pc):
    e = torch.empty
    x = e(0, 64, device="cuda")
    sr.precond_rms_norm(pc.h, x, torch.ones(64, device="cuda"), 1e-6, y=e(0, 64, device="cuda"))
    dw = torch.full((64,), 3.0, device="cuda")
    sr.precond_rms_norm_grad(pc.h, x, x, torch.ones(64, device="cuda"), e(0, device="cuda"), e(0, 64, device="cuda"), dw)
    assert bool((dw == 0).all())
    q, s = sr.empty8(0, 64)
    sr.precond_quantize8(pc.h, x, q=q, scale=s)
    sr.precond_distill(pc.h, e(0, 50, device="cuda"), e(0, 3, dtype=torch.int32, device="cuda"), e(0, 3, device="cuda"), e(0, device="cuda"))
    torch.cuda.synchronize()


def test_launch_count(pc):
    n = sr.precond_launch_count(pc.h)
    x = torch.ones(4, 64, device="cuda")
    sr.precond_rms_norm(pc.h, x, torch.ones(64, device="cuda"), 1e-6, y=torch.empty_like(x))
    assert sr.precond_launch_count(pc.h) == n + 1
