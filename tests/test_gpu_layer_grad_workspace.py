"""Gradients of the layer norm with a workspace of exactly the size that the library asks for: nothing beside it is
written, whatever form the rows take.  (Rows of up to 256 columns that begin at sectors, and many of them, launch the
most blocks.)"""
import pytest
import torch

import shampoo_roots_gb300 as sr
from test_gpu_layer_norm import check_grad, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu
GUARD = 1 << 22


@pytest.mark.parametrize("rows,cols", [(2500, 256), (5000, 128), (10000, 64), (20000, 128), (20000, 256), (6000, 16), (6000, 200), (3000, 257),
                                       (900, 1000), (700, 4096), (300, 9000), (40, 70000), (65, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_beside_the_workspace(pc, rows, cols, dtype):  # noqa: F811
    c = check_grad(pc, rows, cols, dtype, True)
    need = sr.precond_layer_norm_grad_workspace(rows, cols)
    buffer = torch.full((GUARD + need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    d = {k: c[k].cuda() for k in ("x", "dy", "dr", "w", "mean", "rstd")}
    dx, dw, db = (torch.empty_like(c[k]) for k in ("dx", "dw", "db"))
    sr.precond_layer_norm_grad(pc.h, d["dy"], d["x"], d["w"], d["mean"], d["rstd"], dx, dw, db=db, dresidual=d["dr"],
                               workspace=buffer[GUARD:GUARD + need])
    assert bool((buffer[:GUARD] == 0xA5).all()) and bool((buffer[GUARD + need:] == 0xA5).all())
    assert torch.equal(dx, c["dx"]) and torch.equal(dw, c["dw"]) and torch.equal(db, c["db"])
