"""What the operators of a policy's training step refuse, on a host-only handle: arguments are checked before anything
is enqueued (a call that passes them returns ENODEV there), and the binding checks what only it can see."""
import ctypes

import pytest
import torch

import shampoo_roots_gb300 as sr

P = ctypes.c_void_p
BASE = {k: 0x10000000 * (i + 1) for i, k in enumerate("abcdefghijkl")}      # fake, never dereferenced
i64, i32, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_float


@pytest.fixture(scope="module")
def h():
    x = sr.precond_create(-1)
    yield x
    sr.precond_destroy(x)


def norm(kw):
    a = dict(x=BASE["a"], r=BASE["b"], w=BASE["c"], b=BASE["h"], dtype=1, wtype=0, rows=4, cols=256, ldx=256, ldr=256, eps=1e-5,
             total=BASE["d"], ldt=256, y=BASE["e"], ldy=256, q=BASE["f"], ldq=256, s=BASE["g"], mean=BASE["i"], rstd=BASE["j"])
    a.update(kw)
    return sr.load().precond_layer_norm(
        P(a["h_"]), P(a["x"]), P(a["r"]), P(a["w"]), P(a["b"]), i32(a["dtype"]), i32(a["wtype"]), i64(a["rows"]), i64(a["cols"]),
        i64(a["ldx"]), i64(a["ldr"]), f32(a["eps"]), P(a["total"]), i64(a["ldt"]), P(a["y"]), i64(a["ldy"]), P(a["q"]), i64(a["ldq"]),
        P(a["s"]), P(a["mean"]), P(a["rstd"]), P(0))


@pytest.mark.parametrize("bad", [
    dict(h_=None), dict(x=None), dict(w=None), dict(dtype=2), dict(wtype=2), dict(rows=-1), dict(cols=-1), dict(cols=(1 << 30) + 1),
    dict(ldx=255), dict(ldr=1), dict(ldt=255), dict(ldy=0), dict(ldq=264), dict(ldq=240), dict(eps=0.0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(r=None), dict(total=None), dict(q=None), dict(s=None), dict(x=BASE["a"] + 1), dict(b=BASE["h"] + 2),
    dict(wtype=1, b=BASE["h"] + 1), dict(q=BASE["f"] + 8), dict(s=BASE["g"] + 4), dict(mean=BASE["i"] + 2), dict(rstd=BASE["j"] + 1),
    dict(r=None, total=None, y=None, q=None, s=None, mean=None, rstd=None), dict(y=BASE["a"]), dict(y=BASE["d"]), dict(y=BASE["h"]),
    dict(total=BASE["a"], ldt=264), dict(total=BASE["a"] + 512), dict(mean=BASE["j"]), dict(rstd=BASE["h"]), dict(q=BASE["b"])])
def test_norm_refuses(h, bad):
    assert norm({**dict(h_=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(total=BASE["a"]), dict(total=BASE["b"]), dict(r=None, total=None), dict(b=None), dict(y=None),
                                  dict(q=None, s=None), dict(dtype=0), dict(wtype=1), dict(mean=None), dict(rstd=None), dict(rows=0),
                                  dict(cols=0), dict(ldq=512), dict(y=None, q=None, s=None, rstd=None)])
def test_norm_accepts(h, good):
    assert norm({**dict(h_=h), **good}) == sr.ENODEV


def grad(kw):
    a = dict(dy=BASE["a"], x=BASE["b"], w=BASE["c"], mean=BASE["d"], rstd=BASE["e"], dr=BASE["f"], dtype=1, wtype=0, rows=400, cols=256,
             lddy=256, ldx=256, lddr=256, dx=BASE["g"], lddx=256, dw=BASE["h"], db=BASE["i"], ws=BASE["j"], bytes=1 << 20)
    a.update(kw)
    return sr.load().precond_layer_norm_grad(
        P(a["h_"]), P(a["dy"]), P(a["x"]), P(a["w"]), P(a["mean"]), P(a["rstd"]), P(a["dr"]), i32(a["dtype"]), i32(a["wtype"]),
        i64(a["rows"]), i64(a["cols"]), i64(a["lddy"]), i64(a["ldx"]), i64(a["lddr"]), P(a["dx"]), i64(a["lddx"]), P(a["dw"]), P(a["db"]),
        P(a["ws"]), i64(a["bytes"]), P(0))


WIDE = dict(rows=1, cols=32769, lddy=32769, ldx=32769, lddr=32769, lddx=32769)


@pytest.mark.parametrize("bad", [
    dict(h_=None), dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(ws=None),
    dict(bytes=8), dict(ws=BASE["j"] + 4), dict(dtype=2), dict(rows=-1), dict(lddy=255), dict(lddx=255), dict(lddr=3),
    dict(dx=BASE["a"] + 512), dict(dx=BASE["a"], lddx=300), dict(dx=BASE["c"]), dict(dw=BASE["c"]), dict(ws=BASE["a"]), dict(dw=BASE["g"]),
    dict(db=BASE["h"]), dict(db=BASE["i"] + 1), dict(db=BASE["d"]), dict(**WIDE, dx=BASE["a"]), dict(**WIDE, dx=BASE["b"])])
def test_grad_refuses(h, bad):
    assert grad({**dict(h_=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, dict(dr=None), dict(db=None), dict(dx=BASE["a"]), dict(dx=BASE["b"]), dict(dx=BASE["f"]), dict(rows=0),
                                  dict(cols=0), dict(**WIDE)])
def test_grad_accepts(h, good):
    assert grad({**dict(h_=h), **good}) == sr.ENODEV
    assert sr.precond_layer_norm_grad_workspace(-1, 5) == -1 and sr.precond_layer_norm_grad_workspace(0, 5) == 0
    assert sr.precond_layer_norm_grad_workspace(4, 256) == 0 and grad(dict(h_=h, rows=4, ws=None, bytes=0)) == sr.ENODEV   # few rows need none


def policy(kw):
    a = dict(z=BASE["a"], dtype=1, rows=7, vocab=1000, ldz=1000, ids=BASE["b"], bits=32, adv=BASE["c"], old=BASE["d"], ref=BASE["e"],
             weight=BASE["f"], tau=1.0, low=0.2, high=0.2, kl=0.1, loss=BASE["g"], logp=BASE["h"], dz=BASE["i"], lddz=1000)
    a.update(kw)
    return sr.load().precond_policy(
        P(a["h_"]), P(a["z"]), i32(a["dtype"]), i64(a["rows"]), i64(a["vocab"]), i64(a["ldz"]), P(a["ids"]), i32(a["bits"]), P(a["adv"]),
        P(a["old"]), P(a["ref"]), P(a["weight"]), f32(a["tau"]), f32(a["low"]), f32(a["high"]), f32(a["kl"]), P(a["loss"]), P(a["logp"]),
        P(a["dz"]), i64(a["lddz"]), P(0))


SCORE = dict(adv=None, old=None, ref=None, loss=None, dz=None, lddz=0, kl=0.0)


@pytest.mark.parametrize("bad", [
    dict(h_=None), dict(z=None), dict(ids=None), dict(dtype=2), dict(rows=-1), dict(rows=1 << 30), dict(vocab=0), dict(ldz=999),
    dict(lddz=999), dict(bits=16), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-19),
    dict(low=-0.1), dict(low=1.1), dict(low=float("nan")), dict(high=-0.1), dict(high=float("nan")), dict(kl=-1.0), dict(kl=float("inf")),
    dict(kl=float("nan")), dict(ref=None), dict(ids=BASE["b"] + 2), dict(ids=BASE["b"] + 4, bits=64), dict(adv=BASE["c"] + 2),
    dict(old=BASE["d"] + 1), dict(ref=BASE["e"] + 2), dict(weight=BASE["f"] + 1), dict(loss=BASE["g"] + 2), dict(logp=BASE["h"] + 2),
    dict(loss=None, dz=None), dict(adv=None), dict(SCORE, logp=None), dict(SCORE, old=BASE["d"]), dict(SCORE, ref=BASE["e"]),
    dict(SCORE, loss=BASE["g"]), dict(SCORE, dz=BASE["i"], lddz=1000), dict(dz=BASE["a"] + 2), dict(dz=BASE["a"], lddz=1008),
    dict(loss=BASE["a"]), dict(loss=BASE["i"]), dict(logp=BASE["d"]), dict(logp=BASE["g"]), dict(dz=BASE["b"]), dict(loss=BASE["f"])])
def test_policy_refuses(h, bad):
    assert policy({**dict(h_=h), **bad}) == sr.EINVAL


@pytest.mark.parametrize("good", [{}, SCORE, dict(SCORE, weight=None), dict(old=None), dict(ref=None, kl=0.0), dict(kl=0.0), dict(weight=None),
                                  dict(loss=None), dict(logp=None), dict(dz=None, lddz=0), dict(dz=BASE["a"]), dict(bits=64), dict(dtype=0),
                                  dict(high=float("inf")), dict(low=1.0), dict(low=0.0, high=0.0), dict(rows=0)])
def test_policy_accepts(h, good):
    assert policy({**dict(h_=h), **good}) == sr.ENODEV


def make(tensors, dtypes, sizes, count=None):
    """(code, list) of fake tensors."""
    n = len(tensors)
    out = P(1)
    code = sr.load().precond_list_create(ctypes.byref(out), i32(n if count is None else count), (P * max(n, 1))(*tensors),
                                         (ctypes.c_int * max(n, 1))(*dtypes), (i64 * max(n, 1))(*sizes))
    return code, out


@pytest.mark.parametrize("bad", [
    ([None], [0], [4]), ([BASE["a"] + 2], [0], [4]), ([BASE["a"] + 1], [1], [4]), ([BASE["a"]], [2], [4]), ([BASE["a"]], [0], [-1]),
    ([BASE["a"]], [0], [(1 << 44) + 1]), ([BASE["a"], BASE["a"]], [0, 0], [4, 4]), ([BASE["a"], BASE["b"], BASE["a"] + 12], [0, 1, 1], [4, 4, 4]),
    ([BASE["b"], BASE["a"]], [0, 0], [4, 0x4000001]), ([BASE["a"]] * 300, [1] * 300, [1] * 300)])
def test_list_refuses(bad):
    code, out = make(*bad)
    assert code == sr.EINVAL and not out.value


def test_list_refuses_pointers():
    lib = sr.load()
    assert lib.precond_list_create(None, 0, None, None, None) == sr.EINVAL
    assert lib.precond_list_create(ctypes.byref(P()), i32(1), None, None, None) == sr.EINVAL
    assert make([BASE["a"]], [0], [4], count=-1)[0] == sr.EINVAL
    assert lib.precond_list_destroy(None) == sr.OK
    lib.precond_list_workspace.restype = i64
    assert lib.precond_list_workspace(None) == -1


@pytest.mark.parametrize("good", [
    ([], [], []), ([BASE["a"], None], [0, 1], [4, 0]), ([BASE["a"], BASE["a"] + 16], [0, 0], [4, 4]), ([BASE["b"], BASE["a"]], [0, 0], [4, 0x4000000]),
    ([BASE["a"] + 2 * i for i in range(3000)], [1] * 3000, [1] * 3000), ([BASE["a"], BASE["b"]], [0, 1], [1 << 20, 5])])
def test_list_calls(h, good):
    lib = sr.load()
    code, l = make(*good)
    assert code == sr.OK
    lib.precond_list_workspace.restype, lib.precond_list_workspace.argtypes = i64, [P]
    need = lib.precond_list_workspace(l)
    assert need % 8 == 0 and (need > 0) == (sum(good[2]) > 1 << 20 or len(good[0]) > 128)

    def total(hh=h, norm=BASE["k"], ws=BASE["l"], bytes_=need):
        return lib.precond_grad_norm(P(hh), l, P(norm), P(ws), i64(bytes_), P(0))

    def clip(hh=h, most=1.0, norm=BASE["k"], given=0, ws=BASE["l"], bytes_=need):
        return lib.precond_clip_grads(P(hh), l, f32(most), P(norm), i32(given), P(ws), i64(bytes_), P(0))

    assert total() == clip() == clip(most=0.0) == clip(most=float("inf")) == sr.ENODEV
    assert clip(given=1, ws=None, bytes_=0) == sr.ENODEV
    for call in (total, clip):
        for bad in (dict(hh=None), dict(norm=None), dict(norm=BASE["k"] + 2)):
            assert call(**bad) == sr.EINVAL, bad
        for bad in (dict(ws=None), dict(ws=BASE["l"] + 8), dict(bytes_=need - 1), dict(norm=BASE["l"] + 8)):
            assert call(**bad) == (sr.EINVAL if need else sr.ENODEV), bad
        if good[0]:
            assert call(norm=good[0][0]) == sr.EINVAL and call(ws=good[0][0] - 16) == (sr.EINVAL if need else sr.ENODEV)
    for bad in (dict(most=-1.0), dict(most=float("nan"))):
        assert clip(**bad) == sr.EINVAL
    assert lib.precond_list_destroy(l) == sr.OK


def test_binding_refuses(h):
    """Shapes, types and strides, which the library cannot see (CPU tensors: nothing is enqueued)."""
    x, dy = torch.zeros(6, 64), torch.zeros(6, 64)
    w, b, y, m, rs = torch.ones(64), torch.zeros(64), torch.empty(6, 64), torch.empty(6), torch.empty(6)
    q, s = sr.empty8(6, 64, "cpu")
    ok = dict(stream=0, raw=True)
    good = dict(x=x, weight=w, eps=1e-5, bias=b, y=y, q=q, scale=s, mean=m, rstd=rs)
    assert sr.precond_layer_norm(h, **good, **ok) == sr.ENODEV
    for bad in (dict(x=x.double()), dict(x=x[0]), dict(x=x.t()), dict(weight=w[:63]), dict(weight=w.double()), dict(bias=b[:63]),
                dict(bias=b.bfloat16()), dict(y=y[:5]), dict(y=y.bfloat16()), dict(q=q.view(torch.uint8)), dict(scale=None),
                dict(mean=m[:5]), dict(rstd=rs.double()), dict(residual=x[:, :32], total=y), dict(q=None), dict(x=7), dict(weight=3.5)):
        with pytest.raises((TypeError, ValueError, AttributeError, RuntimeError)):
            sr.precond_layer_norm(h, **{**good, **bad}, **ok)
    good = dict(dy=dy, x=x, weight=w, mean=m, rstd=rs, dx=y, dw=torch.empty(64), db=torch.empty(64), workspace=torch.empty(100000))
    assert sr.precond_layer_norm_grad(h, **good, **ok) == sr.ENODEV
    for bad in (dict(x=x.bfloat16()), dict(dy=dy[:5]), dict(mean=m[:5]), dict(db=torch.empty(63)), dict(dw=torch.empty(64, dtype=torch.float64)),
                dict(workspace=torch.empty(64, 64)), dict(dresidual=x[:, :8])):
        with pytest.raises((TypeError, ValueError)):
            sr.precond_layer_norm_grad(h, **{**good, **bad}, **ok)
    z, ids, v = torch.zeros(6, 50), torch.zeros(6, dtype=torch.int64), torch.zeros(6)
    good = dict(logits=z, ids=ids, advantage=v, old_logp=v, weight=v, loss=torch.empty(6), dlogits=z)
    assert sr.precond_policy(h, **good, **ok) == sr.ENODEV
    for bad in (dict(ids=ids.short()), dict(ids=ids[:5]), dict(ids=ids[:, None]), dict(advantage=v.double()), dict(old_logp=v[:5]),
                dict(logits=z.half()), dict(dlogits=z.bfloat16()), dict(loss=torch.empty(5)), dict(weight=v[None]), dict(temperature="1"),
                dict(logp=torch.empty(12)[::2])):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            sr.precond_policy(h, **{**good, **bad}, **ok)
    with pytest.raises(sr.PrecondError):
        sr.precond_policy(h, z, ids, logp=v, stream=0)
    norm = torch.empty(())
    assert sr.precond_grad_norm(h, [x, w], norm, workspace=torch.empty(100000), **ok) == sr.ENODEV
    assert sr.precond_grad_norm(h, [x.t(), torch.zeros(4, 3, 2, 5).permute(2, 0, 3, 1)], norm, workspace=torch.empty(100000), **ok) == sr.ENODEV
    assert sr.precond_clip_grads(h, sr.TensorList([x, w]), 1.0, norm.view(1), given=True, **ok) == sr.ENODEV
    for bad in ([x[:, :32]], [x.half()], [x, x.view(-1)[5:7]], [x, 3], [torch.zeros(3, 4)[:, ::2]], [x.expand(2, 6, 64)]):
        with pytest.raises((TypeError, ValueError, RuntimeError, AttributeError)):
            sr.precond_grad_norm(h, bad, norm, workspace=torch.empty(100000), **ok)
    for bad in (torch.empty(2), torch.empty((), dtype=torch.float64)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            sr.precond_grad_norm(h, [x], bad, workspace=torch.empty(100000), **ok)
    with pytest.raises(TypeError):
        sr.precond_clip_grads(h, [x], "1", norm, **ok)
    l = sr.TensorList(t for t in (x, w))
    assert len(l) == 2 and l.workspace == 0 and l.tensors[0] is x and sr.TensorList([torch.zeros(1 << 20)]).workspace > 0
