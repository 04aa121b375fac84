"""Gradients clipped by their norm over all ranks, between the halves of OwnerSharding.step: two gloo ranks, of which one
owns nothing or a part.  (Plain torch in place of the library's norm and scaling.)"""
import math
import os
import socket

import pytest
import torch

SHAPES = {"one owner": [(6, 4)], "two owners": [(6, 4), (5, 3), (2, 2)]}
MOST = 0.25


def local(rank, shapes):
    g = torch.Generator().manual_seed(rank)
    return [torch.randn(*s, generator=g) for s in shapes]


def _rank(rank, world, port, shapes, q):
    import torch.distributed as dist
    from shampoo_roots_gb300.sharding import OwnerSharding
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        plan = OwnerSharding(shapes, rank, world)
        grads = local(rank, shapes)
        mine = plan.reduce_gradients(grads)
        norm = torch.tensor(math.sqrt(sum(float((g.double() ** 2).sum()) for g in mine)))
        norm.square_()
        dist.all_reduce(norm)
        norm.sqrt_()
        for g in mine:
            g.mul_(min(1.0, MOST / float(norm)))
        out = plan.gather_updates([2 * g for g in mine] if mine else [], device=grads[0].device)
        q.put((rank, float(norm), [o.numpy() for o in out]))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("name", SHAPES)
def test_clipped_by_the_joint_norm(name):
    import torch.multiprocessing as mp
    shapes, world = SHAPES[name], 2
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    port = s.getsockname()[1]
    s.close()
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_rank, args=(r, world, port, shapes, q)) for r in range(world)]
    for p in procs:
        p.start()
    res = [q.get(timeout=120) for _ in range(world)]
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    mean = [(a + b) / 2 for a, b in zip(local(0, shapes), local(1, shapes))]
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in mean))
    assert want > MOST
    for _, norm, out in res:
        assert norm == pytest.approx(want, rel=1e-6)
        for o, g in zip(out, mean):
            assert torch.allclose(torch.from_numpy(o), 2 * g * (MOST / want), rtol=1e-5, atol=0)
