"""What the training-step operators refuse, on a host-only handle: arguments are checked before anything is enqueued
(a call that passes them returns ENODEV there), and the binding checks what only it can see."""
import ctypes

import pytest
import torch

import shampoo_roots_gb300 as sr

P = ctypes.c_void_p
BASE = {k: 0x10000000 * (i + 1) for i, k in enumerate("abcdefghij")}      # fake, never dereferenced


@pytest.fixture(scope="module")
def h():
    x = sr.precond_create(-1)
    yield x
    sr.precond_destroy(x)


def norm(kw):
    a = dict(x=BASE["a"], r=BASE["b"], w=BASE["c"], dtype=1, wtype=0, rows=4, cols=256, ldx=256, ldr=256, eps=1e-6, total=BASE["d"],
             ldt=256, y=BASE["e"], ldy=256, q=BASE["f"], ldq=256, s=BASE["g"], rstd=BASE["i"], stream=0)
    a.update(kw)
    f = sr.load().precond_rms_norm
    i64, i32, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_float
    return f(P(a["h"]), P(a["x"]), P(a["r"]), P(a["w"]), i32(a["dtype"]), i32(a["wtype"]), i64(a["rows"]), i64(a["cols"]), i64(a["ldx"]),
             i64(a["ldr"]), f32(a["eps"]), P(a["total"]), i64(a["ldt"]), P(a["y"]), i64(a["ldy"]), P(a["q"]), i64(a["ldq"]), P(a["s"]),
             P(a["rstd"]), P(a["stream"]))


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(x=None), dict(w=None), dict(dtype=2), dict(dtype=7), dict(wtype=2), dict(rows=-1), dict(cols=-1),
    dict(cols=(1 << 30) + 1), dict(ldx=255), dict(ldr=1), dict(ldt=255), dict(ldy=0), dict(ldq=264), dict(ldq=240), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(r=None), dict(total=None), dict(q=None), dict(s=None), dict(x=BASE["a"] + 1),
    dict(q=BASE["f"] + 8), dict(s=BASE["g"] + 4), dict(rstd=BASE["i"] + 2),
    dict(r=None, total=None, y=None, q=None, s=None, rstd=None),
    dict(y=BASE["a"]), dict(y=BASE["d"]), dict(total=BASE["a"], ldt=264), dict(total=BASE["a"] + 512), dict(total=BASE["c"]),
    dict(q=BASE["a"]), dict(rstd=BASE["d"])])
def test_norm_refuses(h, bad):
    assert norm({**dict(h=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(total=BASE["a"]), dict(total=BASE["b"]), dict(r=None, total=None), dict(y=None), dict(q=None, s=None),
                                  dict(dtype=0), dict(wtype=1), dict(rstd=None), dict(rows=0), dict(cols=0), dict(ldq=512), dict(ldx=1000)])
def test_norm_accepts(h, good):
    assert norm({**dict(h=h), **good}) == sr.ENODEV


def grad(kw):
    a = dict(dy=BASE["a"], x=BASE["b"], w=BASE["c"], rstd=BASE["d"], dr=BASE["e"], dtype=1, wtype=0, rows=4, cols=256, lddy=256, ldx=256,
             lddr=256, dx=BASE["f"], lddx=256, dw=BASE["g"], ws=BASE["i"], bytes=1 << 20)
    a.update(kw)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    return sr.load().precond_rms_norm_grad(
        P(a["h"]), P(a["dy"]), P(a["x"]), P(a["w"]), P(a["rstd"]), P(a["dr"]), i32(a["dtype"]), i32(a["wtype"]), i64(a["rows"]),
        i64(a["cols"]), i64(a["lddy"]), i64(a["ldx"]), i64(a["lddr"]), P(a["dx"]), i64(a["lddx"]), P(a["dw"]), P(a["ws"]), i64(a["bytes"]), P(0))


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(dy=None), dict(x=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(bytes=8),
    dict(ws=BASE["i"] + 4), dict(dtype=2), dict(rows=-1), dict(lddy=255), dict(lddx=255), dict(lddr=3), dict(dx=BASE["a"] + 512),
    dict(dx=BASE["a"], lddx=300), dict(dx=BASE["c"]), dict(dw=BASE["c"]), dict(ws=BASE["a"]), dict(dw=BASE["f"]),
    dict(cols=9000, lddy=9000, ldx=9000, lddr=9000, lddx=9000, dx=BASE["a"])])      # rows read twice: not in place
def test_grad_refuses(h, bad):
    assert grad({**dict(h=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(dr=None), dict(dx=BASE["a"]), dict(dx=BASE["b"]), dict(dx=BASE["e"]), dict(rows=0), dict(cols=0)])
def test_grad_accepts(h, good):
    assert grad({**dict(h=h), **good}) == sr.ENODEV
    assert sr.precond_rms_norm_grad_workspace(-1, 5) == -1 and sr.precond_rms_norm_grad_workspace(0, 5) == 0


def quantize(kw):
    a = dict(x=BASE["a"], dtype=1, rows=300, cols=200, ldx=200, xs=None, block=0, q=BASE["b"], ldq=208, s=BASE["c"], qt=BASE["d"],
             ldqt=304, st=BASE["e"])
    a.update(kw)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    return sr.load().precond_quantize8(P(a["h"]), P(a["x"]), i32(a["dtype"]), i64(a["rows"]), i64(a["cols"]), i64(a["ldx"]), P(a["xs"]),
                                       i32(a["block"]), P(a["q"]), i64(a["ldq"]), P(a["s"]), P(a["qt"]), i64(a["ldqt"]), P(a["st"]), P(0))


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(x=None), dict(dtype=3), dict(dtype=2), dict(xs=BASE["f"]), dict(rows=-2), dict(ldx=199), dict(block=2), dict(block=-1),
    dict(ldq=200), dict(ldq=192), dict(ldqt=288), dict(s=None), dict(q=None), dict(qt=None), dict(q=None, s=None, qt=None, st=None),
    dict(q=BASE["b"] + 1), dict(st=BASE["e"] + 8), dict(q=BASE["a"]), dict(qt=BASE["b"]), dict(st=BASE["c"]),
    dict(dtype=2, xs=BASE["f"], ldx=200), dict(dtype=2, xs=BASE["c"], ldx=208)])
def test_quantize_refuses(h, bad):
    assert quantize({**dict(h=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(block=1), dict(q=None, s=None), dict(qt=None, st=None), dict(dtype=0), dict(rows=0),
                                  dict(dtype=2, xs=BASE["f"], ldx=208)])
def test_quantize_accepts(h, good):
    assert quantize({**dict(h=h), **good}) == sr.ENODEV


def gemm(kw):
    a = dict(m=10, n=20, k=30, a=BASE["a"], lda=32, sa=BASE["b"], b=BASE["c"], ldb=48, sb=BASE["d"], c=BASE["e"], ldc=20, dtype=1, acc=0)
    a.update(kw)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    return sr.load().precond_gemm8(P(a["h"]), i64(a["m"]), i64(a["n"]), i64(a["k"]), P(a["a"]), i64(a["lda"]), P(a["sa"]), P(a["b"]),
                                   i64(a["ldb"]), P(a["sb"]), P(a["c"]), i64(a["ldc"]), i32(a["dtype"]), i32(a["acc"]), P(0))


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(m=-1), dict(k=-1), dict(n=(1 << 30) + 1),
    dict(lda=30), dict(lda=16), dict(ldb=40), dict(ldc=19), dict(dtype=2), dict(dtype=1, acc=1), dict(a=BASE["a"] + 8), dict(sb=BASE["d"] + 1),
    dict(c=BASE["e"] + 1), dict(c=BASE["a"]), dict(c=BASE["b"]), dict(c=BASE["d"] + 256)])
def test_gemm_refuses(h, bad):
    assert gemm({**dict(h=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(dtype=0), dict(dtype=0, acc=1), dict(m=0), dict(k=0), dict(a=BASE["c"], lda=48, sa=BASE["d"])])
def test_gemm_accepts(h, good):
    assert gemm({**dict(h=h), **good}) == sr.ENODEV


def distill(kw):
    a = dict(z=BASE["a"], dtype=1, rows=7, vocab=1000, ldz=1000, ids=BASE["b"], bits=32, ldi=9, t=BASE["c"], ttype=0, ldt=9, top=9,
             weight=BASE["d"], tau=1.0, loss=BASE["e"], dz=BASE["f"], lddz=1000, ws=None, bytes=0)
    a.update(kw)
    i64, i32 = ctypes.c_int64, ctypes.c_int
    return sr.load().precond_distill(P(a["h"]), P(a["z"]), i32(a["dtype"]), i64(a["rows"]), i64(a["vocab"]), i64(a["ldz"]), P(a["ids"]),
                                     i32(a["bits"]), i64(a["ldi"]), P(a["t"]), i32(a["ttype"]), i64(a["ldt"]), i32(a["top"]), P(a["weight"]),
                                     ctypes.c_float(a["tau"]), P(a["loss"]), P(a["dz"]), i64(a["lddz"]), P(a["ws"]), i64(a["bytes"]), P(0))


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(z=None), dict(ids=None), dict(t=None), dict(loss=None), dict(dtype=2), dict(ttype=2), dict(rows=-1), dict(vocab=0),
    dict(ldz=999), dict(lddz=999), dict(ldi=8), dict(ldt=8), dict(bits=16), dict(top=0), dict(top=1025, ldi=1025, ldt=1025), dict(tau=0.0),
    dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(ids=BASE["b"] + 2), dict(weight=BASE["d"] + 1), dict(dz=BASE["a"] + 2),
    dict(dz=BASE["a"], lddz=1008), dict(loss=BASE["a"]), dict(loss=BASE["f"]), dict(loss=BASE["d"]), dict(dz=BASE["b"]),
    dict(rows=2000), dict(rows=2000, ws=BASE["g"], bytes=15999), dict(rows=2000, ws=BASE["g"] + 8, bytes=1 << 20),
    dict(rows=2000, ws=BASE["g"], bytes=16000, dz=BASE["a"]), dict(rows=2000, ws=BASE["a"], bytes=1 << 20)])
def test_distill_refuses(h, bad):
    assert distill({**dict(h=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(weight=None), dict(dz=None, lddz=0), dict(dz=BASE["a"]), dict(bits=64), dict(ttype=1), dict(rows=0),
                                  dict(rows=2000, ws=BASE["g"], bytes=16000), dict(rows=2000, ws=BASE["g"], bytes=1 << 20, dz=BASE["a"])])
def test_distill_accepts(h, good):
    assert distill({**dict(h=h), **good}) == sr.ENODEV


def test_status_and_workspaces(h):
    assert sr.precond_gemm8_status(h, stream=0, raw=True) == sr.ENODEV
    assert sr.load().precond_gemm8_status(None, None) == sr.EINVAL
    assert sr.precond_distill_workspace(4, 100, 5, torch.float32) == 0
    assert sr.precond_distill_workspace(2000, 1000, 5, torch.float32) == 16000
    assert sr.precond_distill_workspace(2000, 1000, 5, torch.float32, True) == 16000 + 2000 * 5 * 4
    assert sr.precond_distill_workspace(2000, 1000, 0, torch.float32) == -1


def test_binding_refuses(h):
    """Shapes, types and strides, which the library cannot see (CPU tensors: nothing is enqueued)."""
    x = torch.zeros(6, 64)
    w, y = torch.ones(64), torch.empty(6, 64)
    q, s = sr.empty8(6, 64, "cpu")
    ok = dict(stream=0, raw=True)
    assert sr.precond_rms_norm(h, x, w, 1e-6, y=y, q=q, scale=s, **ok) == sr.ENODEV
    for bad in (dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(weight=w[:63]), dict(weight=w.double()), dict(y=y[:5]), dict(y=y.bfloat16()),
                dict(q=q.view(torch.uint8)), dict(q=q[:5]), dict(scale=None), dict(scale=s[:, :, :16]), dict(scale=s.float()),
                dict(rstd=torch.empty(5)), dict(rstd=torch.empty(6, dtype=torch.float64)), dict(residual=x[:, :32], total=y), dict(q=None)):
        a = {**dict(x=x, weight=w, eps=1e-6, y=y, q=q, scale=s), **bad}
        with pytest.raises((TypeError, ValueError)):
            sr.precond_rms_norm(h, **a, **ok)
    a, b, c = sr.empty8(6, 64, "cpu"), sr.empty8(9, 64, "cpu"), torch.empty(6, 9)
    assert sr.precond_gemm8(h, *a, *b, c, **ok) == sr.ENODEV
    for bad in ((a[0], a[1], *sr.empty8(9, 65, "cpu"), c), (*a, *b, c.t()), (*a, *b, c.half()), (*a, b[0], a[1][:0], c), (x, a[1], *b, c)):
        with pytest.raises((TypeError, ValueError)):
            sr.precond_gemm8(h, *bad, **ok)
    z, ids, t, loss = torch.zeros(6, 50), torch.zeros(6, 3, dtype=torch.int32), torch.zeros(6, 3), torch.empty(6)
    assert sr.precond_distill(h, z, ids, t, loss, dlogits=z, **ok) == sr.ENODEV
    for bad in ((z, ids.short(), t, loss), (z, ids[:5], t, loss), (z, ids, t[:, :2], loss), (z, ids, t, loss[:5]), (z.half(), ids, t, loss)):
        with pytest.raises((TypeError, ValueError)):
            sr.precond_distill(h, *bad, **ok)
    with pytest.raises((TypeError, ValueError)):
        sr.precond_distill(h, z, ids, t, loss, weight=torch.ones(6, dtype=torch.float64), **ok)
    with pytest.raises((TypeError, ValueError)):
        sr.precond_quantize8(h, x, q=q, scale=s, x_scale=s, **ok)
    with pytest.raises((TypeError, ValueError)):
        sr.precond_quantize8(h, q, q=q, scale=s, **ok)
    with pytest.raises((TypeError, ValueError)):
        sr.precond_quantize8(h, x, qt=q, scale_t=s, **ok)
    with pytest.raises(sr.PrecondError):
        sr.precond_rms_norm(h, x, w, 1e-6, y=y, stream=0)
    with pytest.raises((TypeError, ValueError)):
        sr.precond_rms_norm_grad(h, x, x, w, torch.empty(6), y, torch.empty(64), workspace=torch.empty(64, 64), **ok)


def test_8_bit_helpers():
    """empty8's pitch, scales8 and dequantize8 against the stated layout, byte by byte."""
    rows, cols = 300, 1100
    q, s = sr.empty8(rows, cols, "cpu")
    assert q.shape == (rows, cols) and q.stride() == (1104, 1) and s.shape == sr.scale_shape(rows, cols) == (3, 3, 32, 4, 4)
    flat = s.view(torch.uint8).view(-1)
    flat.copy_(torch.randint(100, 150, flat.shape, dtype=torch.uint8))
    got = sr.scales8(s, rows, cols)
    for r in (0, 1, 31, 32, 127, 128, 200, 299):
        for k in (0, 1, 3, 4, 8):
            at = ((k // 4) * 3 + r // 128) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
            assert float(got[r, k]) == 2.0 ** (int(flat[at]) - 127)
    q.copy_(torch.randn(rows, cols).to(torch.float8_e4m3fn))
    v = sr.dequantize8(q, s)
    assert float(v[299, 1099]) == float(q[299, 1099].float()) * float(got[299, 8])
