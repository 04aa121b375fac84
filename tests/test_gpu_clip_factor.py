"""Clipping where max_norm / norm is below fp32's normal numbers: elements keep their digits.  Tolerances as in
test_gpu_clip.py (the norm 22 E, the factor 2 E, the product E; a second step of the factor E more), and half a step of
the type's smallest numbers, twice in fp32."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_clip import E, E16, TYPES, pc, random  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,most", [(1e28, 1e-16), (3e35, 1e-5), (1e28, 1e-8), (1e36, 3.9), (1e-3, 1e-42), (1e34, 1e-44), (1e28, 0.0), (1.0, 1.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3001, 300007])                         # one cluster; two kernels
def test_small_factors(pc, size, most, dtype, n):  # noqa: F811
    g = P.generator(n)
    most = torch.tensor(most).item()
    held = [random(g, n, dtype, size), random(g, 17, "f32", size)]
    cpu = [t.cpu().double() for t in held]
    norm = torch.empty((), device="cuda")
    sr.precond_grad_norm(pc.h, held, norm)
    exact = math.sqrt(sum(float((c ** 2).sum()) for c in cpu))
    if exact > torch.finfo(torch.float32).max:                       # infinite in fp32: nothing is scaled
        ts = [t.clone() for t in held]
        sr.precond_clip_grads(pc.h, ts, most, norm)
        assert float(norm) == math.inf and all(torch.equal(t, o) for t, o in zip(ts, held))
        return
    assert abs(float(norm) - exact) <= 22 * E * exact
    for given in (False, True):
        ts = [t.clone() for t in held]
        sr.precond_clip_grads(pc.h, ts, most, norm, given=given)
        for t, c in zip(ts, cpu):
            f = c * (most / exact)
            tol = 28 * E * f.abs() + 2.0 ** -149
            if t.dtype == torch.bfloat16:
                tol = tol + E16 * (f.abs() + tol) + 2.0 ** -133
            assert bool(((t.cpu().double() - f).abs() <= tol).all())
