"""The distillation loss where several blocks (a cluster) share a row: 2, 4 and 8 of them, candidates beside the stream
and in a kernel of their own, rows of weight zero between the others, calls one right after the other."""
import pytest
import torch

import shampoo_roots_gb300 as sr
from test_gpu_operators import check_distill, distill_inputs, pc  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,top,dtype", [
    (230, 17000, 20, "f32"),       # 2 blocks a row
    (40, 33001, 20, "f32"),        # 4
    (90, 66000, 300, "bf16"),      # 4, candidates in shared memory
    (21, 70001, 20, "bf16"),       # 8, rows at every alignment
    (1830, 17001, 5, "f32"),       # 2, candidates in a kernel of their own
])
def test_rows_of_a_cluster(pc, rows, vocab, top, dtype):  # noqa: F811
    z, ids, t, w = distill_inputs(rows, vocab, top, dtype)         # every fourth weight is zero
    loss, grad = check_distill(pc, z, ids, t, w, 2.0)
    dz, di, dt, dw = z.cuda(), ids.cuda(), t.cuda(), w.cuda()
    out = [(torch.empty_like(loss), torch.empty_like(grad)) for _ in range(4)]
    for _ in range(5):
        for a, b in out:
            sr.precond_distill(pc.h, dz, di, dt, a, weight=dw, temperature=2.0, dlogits=b)
    for a, b in out:
        assert torch.equal(a, loss) and torch.equal(b, grad)
