"""Temperatures whose square, or whose inverse times log2(e), leaves fp32 gave NaN or 0 for a loss: they are refused."""
import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_operators_refusals import distill, h  # noqa: F401  (h: a host-only handle)


@pytest.mark.parametrize("tau", [1e-40, 4e-39, 1e-25, 9e-19, 1.1e18, 2e19, 1e30, 2.9e38])
def test_refused(h, tau):  # noqa: F811
    assert distill(dict(h=h, tau=tau)) == sr.EINVAL


@pytest.mark.parametrize("tau", [1e-18, 1e-3, 1.0, 50.0, 1e18])
def test_accepted(h, tau):  # noqa: F811
    assert distill(dict(h=h, tau=tau)) == sr.ENODEV


@pytest.mark.gpu
@pytest.mark.parametrize("tau", [1e-18, 1e18])
def test_at_the_ends(tau):
    """One candidate far ahead of the others at both: 1e-18 leaves it alone, and loss = tau (max z - z of it)."""
    pc = sr.Preconditioner(0)
    z = P.randn(P.generator(1), 6, 3000).cuda()
    ids = torch.arange(6, dtype=torch.int32, device="cuda")[:, None] + torch.tensor([[0, 100]], dtype=torch.int32, device="cuda")
    t = torch.tensor([[3.0, 1.0]], device="cuda").expand(6, 2).contiguous()
    loss, grad = torch.empty(6, device="cuda"), torch.empty_like(z)
    sr.precond_distill(pc.h, z, ids, t, loss, temperature=tau, dlogits=grad)
    assert bool(loss.isfinite().all()) and bool(grad.isfinite().all())
    if tau < 1:
        want = tau * (z.double().amax(dim=1) - z.double().gather(1, ids[:, :1].long())[:, 0])
        assert bool(((loss.double() - want).abs() <= 16 * 2.0 ** -24 * want.abs()).all())
    pc.close()
