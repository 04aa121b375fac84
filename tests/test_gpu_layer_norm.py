"""Layer norm and its gradients on the GPU against the plain 64-bit forms (training_plain.py).

Tolerances: E = 2^-24 is fp32's unit roundoff, E16 = 2^-8 bf16's half step.  A row's sums have at most cols / 256 + 64
additions one after another.  The mean is then within `chain` E of the mean magnitude A.  The deviations are taken about
a value that is off by as much; joining the warps' means moves the variance by 2 d(mean) / std of itself at most, so that
rstd, half of it, is within chain E (1 + A / std)."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
import training_plain as T

pytestmark = pytest.mark.gpu
E, E16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def pc():
    p = sr.Preconditioner(0)
    yield p
    p.close()


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu()


def bounds(h, mean, rstd, cols):
    """(of mean, of rstd relative), columns of one a row."""
    f = h.double()
    chain = (cols / 256 + 64) * E
    A = f.abs().mean(dim=1)
    return chain * A, chain * (1 + A * rstd) + 8 * E


def check_norm(pc, rows, cols, dtype, wtype="f32", residual=True, bias=True, pitch=0, offset=0.0, scale=1.0, eps=1e-5):
    g = P.generator(rows * 31 + cols)
    x = (scale * P.randn(g, rows, cols) * torch.exp(P.randn(g, rows, 1)) + offset).to(TYPES[dtype])
    r = (scale * P.randn(g, rows, cols)).to(TYPES[dtype]) if residual else None
    w = (1 + 0.3 * P.randn(g, cols)).to(TYPES[wtype])
    b = (0.5 * P.randn(g, cols)).to(TYPES[wtype]) if bias else None
    place = (lambda t: P.pitched(t, cols + pitch, offset=pitch % 5)) if pitch else (lambda t: t.cuda())
    dx, dr = place(x), place(r) if residual else None
    db = b.cuda() if bias else None
    total = torch.empty_like(x, device="cuda") if residual else None
    y = torch.empty_like(x, device="cuda")
    q, s = sr.empty8(rows, cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sr.precond_layer_norm(pc.h, dx, w.cuda(), eps, bias=db, residual=dr, total=total, y=y, q=q, scale=s, mean=mean, rstd=rstd)
    h, want, m, rs = T.layer_norm(x, r, w, b, eps)
    if residual:
        assert torch.equal(total.cpu(), h)
    tm, tr = bounds(h, m, rs, cols)
    assert bool(((mean.cpu().double() - m).abs() <= tm + 1e-38).all())
    assert bool(((rstd.cpu().double() - rs).abs() <= tr * rs).all())
    # h - mean is off by the mean's error and a rounding; rstd, w, b and the sum by theirs
    n = (want - (0 if b is None else b.double())).abs()
    tol = (tm * rs)[:, None] * w.double().abs() + n * (tr + 4 * E)[:, None] + 2 * E * want.abs() + 1e-38
    assert bool(((y.cpu().double() - want).abs() <= tol + (E16 * (want.abs() + tol) if dtype == "bf16" else 0)).all())
    check8(q, s, want, tol)
    # outputs left out change nothing in the others, unless their rows' places chose another kernel (sums in another order)
    q2, s2 = sr.empty8(rows, cols)
    t2 = torch.empty_like(total) if residual else None
    sr.precond_layer_norm(pc.h, dx, w.cuda(), eps, bias=db, residual=dr, total=t2, q=q2, scale=s2)
    check8(q2, s2, want, tol)
    if not pitch:
        assert torch.equal(bytes_of(q), bytes_of(q2)) and torch.equal(bytes_of(s), bytes_of(s2))
        return
    # every matrix with the same pitch; nothing is written between the rows
    y, total = place(torch.zeros_like(x)), place(torch.zeros_like(x)) if residual else None
    gaps = [(t, t.as_strided((rows - 1, pitch), (cols + pitch, 1), t.storage_offset() + cols)) for t in (y, total) if t is not None]
    held = [gap.clone() for _, gap in gaps]
    sr.precond_layer_norm(pc.h, dx, w.cuda(), eps, bias=db, residual=dr, total=total, y=y, mean=mean, rstd=rstd)
    assert bool(((y.cpu().double() - want).abs() <= tol + (E16 * (want.abs() + tol) if dtype == "bf16" else 0)).all())
    assert bool(((mean.cpu().double() - m).abs() <= tm + 1e-38).all()) and bool(((rstd.cpu().double() - rs).abs() <= tr * rs).all())
    if residual:
        assert torch.equal(total.cpu(), h)
    for (_, gap), was in zip(gaps, held):
        assert torch.equal(bytes_of(gap), bytes_of(was))


def check8(q, s, want, tol):
    """The 8-bit form of a matrix known within tol: the scale fits the block, and each value is a nearest one."""
    rows, cols = want.shape
    sc = sr.scales8(s, rows, cols).cpu().double()
    pad = lambda t: torch.nn.functional.pad(t, (0, P.blocks(cols) * 128 - cols)).view(rows, -1, 128)
    lo, hi = pad((want.abs() - tol).clamp(min=0)).amax(dim=2), pad(want.abs() + tol).amax(dim=2)
    assert bool(((lo <= 448 * sc) & ((hi > 224 * sc) | (lo == 0))).all())
    got = sr.dequantize8(q, s).cpu().double()
    each = sc.repeat_interleave(128, dim=1)[:, :cols]
    assert bool(((got - want).abs() <= torch.maximum((want.abs() + tol) * 2.0 ** -4, each * 2.0 ** -10) + tol).all())
    order = P.order_scales(torch.zeros(rows, P.blocks(cols), dtype=torch.int64), rows, cols)
    assert bool((bytes_of(s).view(-1)[order == 127] == 127).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2), (1, 64), (1, 1024), (3, 100), (5, 128), (130, 256), (257, 1000), (33, 4096),
                                       (17, 4104), (9, 6144), (7, 8200), (5, 16384), (3, 16392), (2, 40000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm(pc, rows, cols, dtype):
    check_norm(pc, rows, cols, dtype)
    check_norm(pc, rows, cols, dtype, wtype="bf16", residual=False, bias=False)


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(500, 48, "bf16", 0), (77, 130, "bf16", 14), (301, 256, "f32", 0), (40, 7001, "bf16", 0),
                                                   (90, 6146, "f32", 6), (77, 13001, "bf16", 1), (50, 24577, "f32", 0), (45, 49153, "bf16", 0),
                                                   (700, 1213, "bf16", 0), (330, 2009, "f32", 0), (200, 530, "bf16", 1), (3, 70000, "f32", 0),
                                                   (19, 72, "bf16", 3), (19, 1001, "f32", 8), (2000, 513, "f32", 3), (6, 65537, "bf16", 0)])
def test_norm_layouts(pc, rows, cols, dtype, pitch):
    """Several rows in a warp, rows at every alignment, rows shared by 2, 4 and 8 blocks and longer ones; more rows than run at once."""
    check_norm(pc, rows, cols, dtype, pitch=pitch)
    check_norm(pc, rows, cols, dtype, wtype="bf16", residual=False, pitch=pitch)


@pytest.mark.parametrize("cols", [100, 3000, 9000, 20001, 70000])
@pytest.mark.parametrize("offset,scale", [(1000.0, 1.0), (-3e4, 0.1), (0.0, 1e-12), (0.0, 1e15)])
def test_norm_far_from_zero(pc, cols, offset, scale):
    """Means a thousand and more standard deviations away: no difference of large sums."""
    check_norm(pc, 21, cols, "f32", residual=False, offset=offset, scale=scale)


def test_norm_one_large_column(pc):
    """A column that is all of the variance, the first and the last."""
    for at in (0, 799):
        x = P.randn(P.generator(at), 9, 800)
        x[:, at] = 3e5
        y, m, r = torch.empty(9, 800, device="cuda"), torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        w = torch.ones(800)
        sr.precond_layer_norm(pc.h, x.cuda(), w.cuda(), 1e-5, y=y, mean=m, rstd=r)
        _, want, mean, rstd = T.layer_norm(x, None, w, None, 1e-5)
        tm, tr = bounds(x, mean, rstd, 800)
        assert bool(((m.cpu().double() - mean).abs() <= tm).all()) and bool(((r.cpu().double() - rstd).abs() <= tr * rstd).all())


def test_norm_values(pc):
    """Rows of one value (no variance), a NaN and an infinity; the neighbours keep their values."""
    x = P.randn(P.generator(1), 40, 512)
    x[3], x[5] = 0, -7.25
    x[7, 100] = math.nan
    x[9, 5] = math.inf
    w, b = torch.ones(512), torch.linspace(-1, 1, 512)
    y = torch.empty(40, 512, device="cuda")
    q, s = sr.empty8(40, 512)
    m, r = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    sr.precond_layer_norm(pc.h, x.cuda(), w.cuda(), 1e-5, bias=b.cuda(), y=y, q=q, scale=s, mean=m, rstd=r)
    _, want, mean, rstd = T.layer_norm(x, None, w, b, 1e-5)
    y, d = y.cpu(), sr.dequantize8(q, s).cpu()
    assert torch.equal(y[3], b) and torch.equal(y[5], b) and float(m[5]) == -7.25
    assert abs(float(r[5]) - 1e-5 ** -0.5) <= 1e-5 ** -0.5 * 8 * E
    assert bool(y[7].isnan().all()) and bool(d[7].isnan().all()) and bool(y[9].isnan().all())
    keep = torch.ones(40, dtype=torch.bool)
    keep[[7, 9]] = False
    tm, tr = bounds(x, mean, rstd, 512)
    tol = (tm * rstd)[:, None] + (want - b.double()).abs() * (tr + 4 * E)[:, None] + 2 * E * want.abs()
    assert bool(((y.double() - want).abs() <= tol)[keep].all())


@pytest.mark.parametrize("rows,cols", [(21, 200), (21, 1000), (21, 20000), (21, 70000), (1500, 2048), (400, 9000)])
def test_norm_in_place(pc, rows, cols):
    g = P.generator(3)
    x, r = P.randn(g, rows, cols), P.randn(g, rows, cols)
    w = torch.ones(cols, device="cuda")
    for over in ("x", "residual"):
        dx, dr = x.cuda(), r.cuda()
        y, y2, t = (torch.empty(rows, cols, device="cuda") for _ in range(3))
        sr.precond_layer_norm(pc.h, dx, w, 1e-6, residual=dr, total=t, y=y)
        sr.precond_layer_norm(pc.h, dx, w, 1e-6, residual=dr, total=dx if over == "x" else dr, y=y2)
        assert torch.equal(t, dx if over == "x" else dr) and torch.equal(y, y2)


def check_grad(pc, rows, cols, dtype, residual, pitch=0, wtype="f32"):
    g = P.generator(rows * 77 + cols)
    x = (P.randn(g, rows, cols) + P.randn(g, rows, 1)).to(TYPES[dtype])
    dy = (P.randn(g, rows, cols) * torch.exp(2 * P.randn(g, rows, 1))).to(TYPES[dtype])
    dr = P.randn(g, rows, cols).to(TYPES[dtype]) if residual else None
    w = (1 + 0.3 * P.randn(g, cols)).to(TYPES[wtype])
    _, _, mean, rstd = T.layer_norm(x, None, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    place = (lambda t: P.pitched(t, cols + pitch, offset=pitch % 5)) if pitch else (lambda t: t.cuda())
    dx = torch.full((rows, cols), math.nan, device="cuda").to(TYPES[dtype])
    dw, db = (torch.full((cols,), math.nan, device="cuda") for _ in range(2))
    args = (place(dy), place(x), w.cuda(), mean.cuda(), rstd.cuda())
    d_dr = place(dr) if residual else None
    sr.precond_layer_norm_grad(pc.h, *args, dx, dw, db=db, dresidual=d_dr)
    wx, ww, wb = T.layer_norm_grad(dy, x, w, mean, rstd, dr)
    f = lambda t: t.double()
    n = ((f(x) - f(mean)[:, None]) * f(rstd)[:, None]).abs()
    gw = (f(dy) * f(w)).abs()
    over = lambda t: t.mean(dim=1, keepdim=True)
    size = f(rstd)[:, None] * (gw + over(gw) + n * over(gw * n)) + (f(dr).abs() if residual else 0)
    tol = (cols / 32 + 24) * E * size + 1e-38
    assert bool(((dx.cpu().double() - wx).abs() <= tol + (E16 * (wx.abs() + tol) if dtype == "bf16" else 0)).all())
    chain = (rows / 8 + 48) * E
    assert bool(((dw.cpu().double() - ww).abs() <= chain * (f(dy).abs() * n).sum(dim=0) + 1e-38).all())
    assert bool(((db.cpu().double() - wb).abs() <= chain * f(dy).abs().sum(dim=0) + 1e-38).all())
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)             # without db the others are the same
    sr.precond_layer_norm_grad(pc.h, *args, dx2, dw2, dresidual=d_dr)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    if pitch:                                                         # every matrix with the same pitch
        dx3 = place(torch.zeros_like(x))
        sr.precond_layer_norm_grad(pc.h, *args, dx3, dw2, db=db, dresidual=d_dr)
        assert bool(((dx3.cpu().double() - wx).abs() <= tol + (E16 * (wx.abs() + tol) if dtype == "bf16" else 0)).all())
        assert bool(((dw2.cpu().double() - ww).abs() <= chain * (f(dy).abs() * n).sum(dim=0) + 1e-38).all())
        assert bool(((db.cpu().double() - wb).abs() <= chain * f(dy).abs().sum(dim=0) + 1e-38).all())
    return dict(x=x, dy=dy, dr=dr, w=w, mean=mean, rstd=rstd, dx=dx, dw=dw, db=db)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (2, 1024), (300, 100), (1000, 256), (77, 1000), (40, 4096), (33, 4104),
                                       (9, 8192), (7, 8200), (5, 20000), (3, 70000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grad(pc, rows, cols, dtype):
    check_grad(pc, rows, cols, dtype, True)
    check_grad(pc, rows, cols, dtype, False, wtype="bf16")


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(3000, 48, "bf16", 0), (77, 130, "bf16", 14), (1001, 256, "f32", 0), (200, 9001, "bf16", 0),
                                                   (190, 6146, "f32", 6), (77, 17000, "bf16", 8), (50, 24577, "f32", 0), (45, 49153, "bf16", 1),
                                                   (2000, 1213, "bf16", 0), (600, 2009, "f32", 0), (900, 530, "bf16", 1), (2500, 384, "f32", 0),
                                                   (19, 1001, "bf16", 3), (5, 65537, "bf16", 0), (300, 5000, "bf16", 0)])
def test_grad_layouts(pc, rows, cols, dtype, pitch):
    check_grad(pc, rows, cols, dtype, True, pitch=pitch)
    check_grad(pc, rows, cols, dtype, False, pitch=pitch)


@pytest.mark.parametrize("cols,dtype", [(640, "bf16"), (1001, "f32"), (20000, "bf16"), (32768, "f32")])
def test_grad_in_place(pc, cols, dtype):
    c = check_grad(pc, 50, cols, dtype, True)
    for over in ("dy", "dr", "x"):
        d = {k: c[k].cuda() for k in ("x", "dy", "dr", "w", "mean", "rstd")}
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        sr.precond_layer_norm_grad(pc.h, d["dy"], d["x"], d["w"], d["mean"], d["rstd"], d[over], dw, db=db, dresidual=d["dr"])
        assert torch.equal(d[over], c["dx"]) and torch.equal(dw, c["dw"]) and torch.equal(db, c["db"])


def test_grad_against_differences(pc):
    """<dx, u>, <dw, v> and <db, v> against central differences of the 64-bit norm along random directions."""
    g = P.generator(12)
    rows, cols, eps = 6, 300, 1e-3
    x, dy, w, b = P.randn(g, rows, cols) + 2, P.randn(g, rows, cols), 1 + 0.3 * P.randn(g, cols), P.randn(g, cols)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sr.precond_layer_norm(pc.h, x.cuda(), w.cuda(), eps, bias=b.cuda(), mean=mean, rstd=rstd)
    dx, dw, db = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    sr.precond_layer_norm_grad(pc.h, dy.cuda(), x.cuda(), w.cuda(), mean, rstd, dx, dw, db=db)
    f = lambda a, c, e: float((T.layer_norm(a, None, c, e, eps)[1] * dy.double()).sum())
    x, w, b, step = x.double(), w.double(), b.double(), 1e-5
    for _ in range(4):
        u, v = P.randn(g, rows, cols).double(), P.randn(g, cols).double()
        along = ((f(x + step * u, w, b) - f(x - step * u, w, b)) / (2 * step), (f(x, w + step * v, b) - f(x, w - step * v, b)) / (2 * step),
                 (f(x, w, b + step * v) - f(x, w, b - step * v)) / (2 * step))
        # differences of an fp64 sum of about 50: step^2 and 1e-16 * 50 / step, both below 1e-7
        for got, want, k in zip((dx, dw, db), along, (u, v, v)):
            assert abs(float((got.cpu().double() * k).sum()) - want) <= 1e-4


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(700, 6144, "bf16", 0), (2600, 1000, "bf16", 0), (5000, 264, "bf16", 0), (2450, 512, "f32", 0),
                                                   (400, 16384, "bf16", 0), (310, 8200, "bf16", 8), (333, 9004, "f32", 4), (1000, 4104, "f32", 8),
                                                   (2000, 1208, "bf16", 24), (320, 12288, "bf16", 0), (1500, 2052, "f32", 12),
                                                   (3700, 65, "bf16", 0), (3000, 200, "bf16", 0), (2500, 333, "f32", 0), (2500, 777, "bf16", 2),
                                                   (700, 6143, "bf16", 0), (900, 4097, "f32", 1), (330, 10001, "bf16", 0), (320, 9001, "f32", 3),
                                                   (340, 16383, "bf16", 0), (5000, 130, "f32", 5), (1000, 3001, "bf16", 7),
                                                   (310, 8200, "bf16", 40), (2000, 1004, "f32", 20), (900, 5000, "bf16", 40), (320, 15008, "bf16", 0),
                                                   (330, 9996, "f32", 60), (170, 13012, "f32", 20)])
def test_norm_many_rows(pc, rows, cols, dtype, pitch):
    """Enough rows for each group of threads to have several: rows copied through shared memory, more than its ring holds."""
    check_norm(pc, rows, cols, dtype, pitch=pitch)
    check_norm(pc, rows, cols, dtype, wtype="bf16", residual=False, pitch=pitch, offset=3.0)


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(700, 4096, "bf16", 0), (2600, 1000, "bf16", 0), (2700, 264, "bf16", 0), (2450, 512, "f32", 0),
                                                   (400, 8192, "bf16", 0), (333, 6148, "f32", 4), (1000, 3004, "f32", 4), (2000, 1208, "bf16", 24),
                                                   (200, 8192, "f32", 0), (3000, 2056, "bf16", 8), (3700, 65, "bf16", 0), (3000, 200, "bf16", 0),
                                                   (2600, 333, "f32", 0), (2500, 777, "bf16", 2), (400, 8191, "bf16", 0), (900, 4097, "f32", 1),
                                                   (5000, 130, "f32", 5), (1000, 3001, "bf16", 7), (400, 6001, "f32", 2),
                                                   (700, 4104, "bf16", 40), (1500, 3004, "f32", 20), (200, 8184, "bf16", 40), (2000, 1000, "bf16", 40)])
def test_grad_many_rows(pc, rows, cols, dtype, pitch):
    check_grad(pc, rows, cols, dtype, True, pitch=pitch)
    c = check_grad(pc, rows, cols, dtype, False, pitch=pitch)
    d = {k: c[k].cuda() for k in ("x", "dy", "w", "mean", "rstd")}
    dw = torch.empty(cols, device="cuda")
    sr.precond_layer_norm_grad(pc.h, d["dy"], d["x"], d["w"], d["mean"], d["rstd"], d["dy"], dw)
    assert torch.equal(d["dy"], c["dx"]) and (pitch or torch.equal(dw, c["dw"]))


@pytest.mark.parametrize("rows,cols,dtype,pitch", [(r, c, d, 0) for r in (1, 8, 9, 17, 60, 190) for c, d in ((200, "bf16"), (1000, "f32"), (1001, "bf16"))]
                         + [(24, 64, "f32", 0), (25, 5000, "bf16", 0), (3, 6000, "f32", 0), (384, 128, "bf16", 0), (24, 6100, "f32", 3)])
def test_grad_few_rows(pc, rows, cols, dtype, pitch):
    """Rows that one block, or a cluster of 2, 4 or 8, takes alone; and just more than that."""
    check_grad(pc, rows, cols, dtype, True, pitch=pitch)
    check_grad(pc, rows, cols, dtype, False, pitch=pitch, wtype="bf16")


def test_empty_and_streams(pc):
    """No rows and no columns; another stream; a captured call replayed on new values."""
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    sr.precond_layer_norm(pc.h, e, w, 1e-5, y=torch.empty_like(e), mean=torch.empty(0, device="cuda"))
    dw, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    z = torch.empty(0, device="cuda")
    sr.precond_layer_norm_grad(pc.h, e, e, w, z, z, torch.empty_like(e), dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    e = torch.empty(5, 0, device="cuda")
    sr.precond_layer_norm(pc.h, e, w[:0], 1e-5, y=torch.empty_like(e))
    x = torch.randn(300, 1500, device="cuda")
    w, dy = torch.randn(1500, device="cuda"), torch.randn(300, 1500, device="cuda")
    out = {k: torch.empty(300, 1500, device="cuda") for k in ("y", "dx")}
    m, r, dw, db = (torch.empty(n, device="cuda") for n in (300, 300, 1500, 1500))
    ws = torch.empty(sr.precond_layer_norm_grad_workspace(300, 1500), dtype=torch.uint8, device="cuda")

    def both(stream=None):
        sr.precond_layer_norm(pc.h, x, w, 1e-5, y=out["y"], mean=m, rstd=r, stream=stream)
        sr.precond_layer_norm_grad(pc.h, dy, x, w, m, r, out["dx"], dw, db=db, workspace=ws, stream=stream)
        return [t.clone() for t in (out["y"], out["dx"], dw, db, m, r)]

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    with pytest.raises(ValueError):
        sr.precond_layer_norm_grad(pc.h, dy, x, w, m, r, out["dx"], dw, stream=side)
    with torch.cuda.stream(torch.cuda.default_stream()):
        torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(torch.randn(300, 1500, device="cuda") * 3 + 1)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [t.clone() for t in got]
    for a, b in zip(replayed, both()):
        assert torch.equal(a, b)


def test_devices_are_not_mixed(pc):
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64)
    with pytest.raises(ValueError):
        sr.precond_layer_norm(pc.h, x, w, 1e-5, y=torch.empty_like(x))
    with pytest.raises(ValueError):
        sr.precond_policy(pc.h, x, torch.zeros(4, dtype=torch.int64), logp=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        sr.precond_grad_norm(pc.h, [x, w], torch.empty((), device="cuda"))
    with pytest.raises(ValueError):
        sr.precond_grad_norm(pc.h, [x], torch.empty(()))
