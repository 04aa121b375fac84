"""The norm of a list of gradients, and their clipping, on the GPU against 64 bits (training_plain.py).

Tolerances: E = 2^-24.  At most 33 squares are added in a row in fp32, everything above them in pairs; with the squares'
own rounding the norm, half of it, is within 20 E, and its fp32 value E more.  The factor is within 2 E of that,
and a scaled element is rounded to fp32 and then to its type."""
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


def check(pc, tensors, share=0.5, scale=None):
    """tensors: on the device; the norm, clipping at `share` of it, and clipping where nothing is to be done."""
    cpu = [t.cpu() for t in tensors]
    want = T.grad_norm(cpu)
    norm, again = torch.full((), math.nan, device="cuda"), torch.full((), math.nan, device="cuda")
    lst = sr.TensorList(tensors)
    sr.precond_grad_norm(pc.h, lst, norm)
    if want > torch.finfo(torch.float32).max:       # 40000 elements of 3e37 have a norm of 6e39: infinite in fp32
        sr.precond_clip_grads(pc.h, lst, 1.0, again)
        assert float(norm) == float(again) == math.inf and all(torch.equal(t.cpu(), c) for t, c in zip(tensors, cpu))
        return
    assert abs(float(norm) - want) <= 22 * E * want
    sr.precond_clip_grads(pc.h, lst, max(want * 1.001, 1e-30), again)
    assert torch.equal(norm, again)
    for t, c in zip(tensors, cpu):
        assert torch.equal(t.cpu(), c)
    again.fill_(math.nan)
    most = share * want
    sr.precond_clip_grads(pc.h, lst, most, again)
    assert torch.equal(norm, again)
    if want == 0:
        return
    # max_norm goes to fp32 on its way
    for t, c in zip(tensors, cpu):
        f = c.double() * share
        tol = 28 * E * f.abs() + 2.0 ** -149
        if t.dtype == torch.bfloat16:
            tol = tol + E16 * (f.abs() + tol) + 2.0 ** -133
        assert bool(((t.cpu().double() - f).abs() <= tol).all())


def random(gen, n, dtype, size=1e-3):
    return (size * P.randn(gen, n)).to(TYPES[dtype]).cuda()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 255, 1000, 8191, 8192, 8193, 70001, 1000003])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_tensor(pc, n, dtype):
    check(pc, [random(P.generator(n), n, dtype)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_alignment(pc, dtype):
    """Views at each element offset of one buffer, beside one another; what lies between them keeps its values."""
    g = P.generator(3)
    buf = random(g, 60000, dtype)
    views, at = [], 1
    for i in range(40):
        n = 1 + (i * 397) % 1500
        views.append(buf[at:at + n])
        at += n + (i % 5)
    held = buf.clone()
    mask = torch.ones(60000, dtype=torch.bool, device="cuda")
    for v in views:
        o = (v.data_ptr() - buf.data_ptr()) // buf.element_size()
        mask[o:o + v.numel()] = False
    check(pc, views)
    assert torch.equal(buf[mask], held[mask])


@pytest.mark.parametrize("count", [2, 31, 32, 33, 224, 225, 1400, 1401, 3000])
def test_many_tensors(pc, count):
    """Both types, empty and one-element tensors among them; more than go into one launch."""
    g = P.generator(count)
    tensors = []
    for i in range(count):
        n = 0 if i % 11 == 3 else 1 if i % 7 == 2 else 1 + (i * 7919) % 3000
        tensors.append(random(g, n, "bf16" if i % 3 else "f32", size=10.0 ** (i % 4 - 3)))
    if count < 3:
        tensors = [random(g, 5000, "bf16"), random(g, 40001, "f32")]
    check(pc, tensors)


def test_shapes(pc):
    """Any dimensions, dense in any order; numbers without a dimension; a sequence of tensors in place of a list."""
    g = P.generator(5)
    t = [random(g, 4 * 6 * 8, "f32").view(4, 6, 8).permute(2, 0, 1), random(g, 300, "bf16").view(20, 15).t(), random(g, 1, "f32").view(())]
    check(pc, t)
    norm, same = torch.empty(1, device="cuda"), torch.empty((), device="cuda")
    sr.precond_grad_norm(pc.h, t, norm)
    sr.precond_grad_norm(pc.h, iter(t), same)
    assert float(norm) == float(same)
    for empty in ([], [torch.empty(0, device="cuda")], [torch.empty(3, 0, device="cuda", dtype=torch.bfloat16)]):
        norm.fill_(7)
        sr.precond_grad_norm(pc.h, empty, norm)
        assert float(norm) == 0
        norm.fill_(7)
        sr.precond_clip_grads(pc.h, empty, 0.5, norm)
        assert float(norm) == 0
    norm.fill_(3.0)
    sr.precond_clip_grads(pc.h, [], 0.5, norm, given=True)
    assert float(norm) == 3.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_values(pc, dtype):
    """Elements whose squares overflow or vanish in fp32, alone and beside ordinary ones; zeros; the smallest numbers."""
    g = P.generator(6)
    for size in (1e-30, 1e-38, 1e25, 3e37, 1e-10):
        check(pc, [random(g, 40000, dtype, size)])
    one = torch.zeros(50000, dtype=TYPES[dtype], device="cuda")
    check(pc, [one])
    for at in (0, 3, 25000, 49999):
        t = one.clone()
        t[at] = 1e-39
        check(pc, [t, one.clone()])
        t = random(g, 50000, dtype)
        t[at] = 1e22
        check(pc, [t])
    check(pc, [random(g, 3000, dtype, 1e30), random(g, 3000, "f32", 1e-30)])
    # sums of each range beside one another: many small beside one ordinary, many ordinary beside one large
    check(pc, [random(g, 400000, dtype, 1e-12), random(g, 5, "f32", 3e-11)])
    check(pc, [random(g, 400000, dtype, 5e11), random(g, 7, "f32", 3e12), random(g, 1, dtype, 1e-3)])
    check(pc, [random(g, 100, dtype, 1e-12), random(g, 100, "f32", 1.0), random(g, 100, dtype, 1e13)])


def test_not_finite(pc):
    """A norm that is not finite leaves the gradients as they are."""
    for bad in (math.nan, math.inf, -math.inf):
        for dtype in ("bf16", "f32"):
            for at in (0, 700, 4999):
                t, u = random(P.generator(at), 5000, dtype), random(P.generator(1), 100, "f32")
                t[at] = bad
                held, norm = t.clone(), torch.zeros((), device="cuda")
                keep = u.clone()
                sr.precond_clip_grads(pc.h, [u, t], 1e-6, norm)
                assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
                assert torch.equal(t.view(torch.uint8), held.view(torch.uint8)) and torch.equal(u, keep)
    t = torch.full((1000,), 3e38, device="cuda")                     # finite elements, a norm beyond fp32
    norm = torch.zeros((), device="cuda")
    sr.precond_clip_grads(pc.h, [t], 1.0, norm)
    assert float(norm) == math.inf and bool((t == torch.tensor(3e38).item()).all())
    norm.fill_(math.nan)
    t = random(P.generator(2), 1000, "f32")
    held = t.clone()
    for given in (math.nan, math.inf, 0.0, 0.5):
        norm.fill_(given)
        sr.precond_clip_grads(pc.h, [t], 0.5, norm, given=True)
        assert torch.equal(t, held)


def test_given_norm(pc):
    """The norm of two lists (two ranks' shares, say), each clipped by it."""
    g = P.generator(9)
    one, two = [random(g, 5000, "bf16"), random(g, 77, "f32")], [random(g, 9001, "f32")]
    cpu = [t.cpu().double() for t in one + two]
    norms = torch.empty(2, device="cuda")
    sr.precond_grad_norm(pc.h, one, norms[0])
    sr.precond_grad_norm(pc.h, two, norms[1])
    norm = norms.square().sum().sqrt()
    want = T.grad_norm(cpu)
    assert abs(float(norm) - want) <= 26 * E * want
    sr.precond_clip_grads(pc.h, one, 0.25 * want, norm, given=True)
    sr.precond_clip_grads(pc.h, two, 0.25 * want, norm, given=True)
    for t, c in zip(one + two, cpu):
        f = 0.25 * c
        tol = 32 * E * f.abs()
        assert bool(((t.cpu().double() - f).abs() <= tol + (E16 * (f.abs() + tol) if t.dtype == torch.bfloat16 else 0)).all())


def test_limits(pc):
    t = random(P.generator(4), 3000, "f32")
    held, norm = t.clone(), torch.empty((), device="cuda")
    sr.precond_clip_grads(pc.h, [t], math.inf, norm)
    assert torch.equal(t, held)
    sr.precond_clip_grads(pc.h, [t], float(norm), norm)               # at the bound nothing is scaled
    assert torch.equal(t, held)
    sr.precond_clip_grads(pc.h, [t], 0.0, norm)
    assert bool((t == 0).all()) and float(norm) > 0


def test_large(pc):
    """A list of 1.2 GB, and a tensor of more than 2^31 elements: offsets beyond 32 bits; the same sum on every call."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    t = torch.empty(2 ** 31 + 12345, dtype=torch.bfloat16, device="cuda")
    t.fill_(2.0 ** -9)
    t[-1], t[2 ** 31 + 7] = 3.0, -5.0
    norm, again = torch.empty((), device="cuda"), torch.empty((), device="cuda")
    sr.precond_grad_norm(pc.h, [t[1:]], norm)
    want = math.sqrt((2 ** 31 + 12342) * 2.0 ** -18 + 34.0)
    assert abs(float(norm) - want) <= 22 * E * want
    sr.precond_clip_grads(pc.h, [t[1:]], 0.5 * want, again)
    assert torch.equal(norm, again)
    assert float(t[0]) == 2.0 ** -9 and float(t[1]) == 2.0 ** -10 and float(t[-1]) == 1.5 and float(t[2 ** 31 + 7]) == -2.5
    assert bool((t[2 ** 30:2 ** 30 + 4096] == 2.0 ** -10).all()) and bool((t[-12340:-12338] == 2.0 ** -10).all())
    del t
    big = [torch.randn(5000, 5003, generator=g, device="cuda") for _ in range(12)]
    sr.precond_grad_norm(pc.h, big, norm)
    sr.precond_grad_norm(pc.h, big, again)
    assert torch.equal(norm, again)
    want = math.sqrt(sum(float(x.double().square().sum()) for x in big))
    assert abs(float(norm) - want) <= 22 * E * want
    held = [x.clone() for x in big]
    sr.precond_clip_grads(pc.h, big, 0.5 * want, norm)
    for x, y in zip(big, held):
        assert bool(((x - 0.5 * y).abs() <= 32 * E * y.abs()).all())


def test_captured_and_two_streams(pc):
    """Two captured calls, each with a workspace of its own, replayed side by side; the list is gone by then."""
    sets = [[random(P.generator(i), 300000 + i, "bf16"), random(P.generator(i + 9), 7001, "f32")] for i in range(2)]
    held = [[t.clone() for t in s] for s in sets]
    norms = torch.zeros(2, device="cuda")
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    sr.precond_grad_norm(pc.h, sets[0], norms[0])
    for s, i, st in zip(sets, range(2), streams):
        lst = sr.TensorList(s)
        ws = torch.empty(lst.workspace, dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sr.precond_clip_grads(pc.h, lst, 0.01, norms[i], workspace=ws)
        graphs.append((gr, ws))
        del lst
    torch.cuda.synchronize()
    for _ in range(3):
        for s, h in zip(sets, held):
            for t, c in zip(s, h):
                t.copy_(c)
        torch.cuda.synchronize()
        for (gr, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for i, (s, h) in enumerate(zip(sets, held)):
            want = T.grad_norm([t.cpu() for t in h])
            assert abs(float(norms[i]) - want) <= 22 * E * want
            f = h[1].cpu().double() * (0.01 / want)
            assert bool(((s[1].cpu().double() - f).abs() <= 28 * E * f.abs()).all())
