"""The training-step operators at sizes that reach every kernel and every turn of its loops: more rows than run at once,
rows too long for registers, products of several tiles a pair of blocks whose ring and scale buffers turn over, large
vocabularies, candidates in a kernel of their own.  The plain forms are in 64 bits (of the large cases on the GPU).

Beside each size stands what the shape rules of the host side make of it on 152 SMs."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_operators import (E16, E32, TYPES, bytes_of, check_distill, check_grad, check_norm,  # noqa: F401
                                distill_inputs, pc)

pytestmark = pytest.mark.gpu
F64 = torch.float64


# ------------------------------------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows,cols", [(5000, 640),      # several rows a block, 4 to 5 turns
                                       (7000, 1024), (2000, 4096), (1000, 6144),   # whole warps of one block a row, 3 to 13 turns
                                       (1000, 8192), (500, 16384),   # 32 columns a thread; gradients: 2 and 4 blocks a row
                                       (400, 24576)])    # 4 blocks a row
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_aligned_rows_beyond_the_grid(pc, rows, cols, dtype):  # noqa: F811
    check_norm(pc, rows, cols, dtype, "f32", True)
    check_norm(pc, rows, cols, dtype, "bf16", False)
    check_grad(pc, rows, cols, dtype, True)
    check_grad(pc, rows, cols, dtype, False)


@pytest.mark.parametrize("rows,cols,dtype", [(200, 49168, "f32"), (200, 50001, "f32"), (200, 50000, "bf16"), (180, 50001, "bf16")])
def test_rows_read_twice_norm(pc, rows, cols, dtype):  # noqa: F811
    check_norm(pc, rows, cols, dtype, "f32", True)
    check_norm(pc, rows, cols, dtype, "bf16", False)


@pytest.mark.parametrize("rows,cols,dtype", [(200, 49168, "f32"), (200, 50001, "f32"), (200, 66000, "bf16"), (320, 66001, "bf16"),
                                             (3, 70000, "f32")])
def test_rows_read_twice_gradients(pc, rows, cols, dtype):  # noqa: F811
    check_grad(pc, rows, cols, dtype, True)
    check_grad(pc, rows, cols, dtype, False)


# ------------------------------------------------------------------------------------------------ product
def random8(gen, rows, cols):
    """A matrix in 8-bit form of random bytes and scales of 2^-3 .. 2^3, and its values."""
    b = torch.randint(0, 256, (rows, cols), generator=gen, dtype=torch.uint8)
    b[(b & 127) == 127] = 0
    e = torch.randint(124, 131, (rows, P.blocks(cols)), generator=gen)
    q, s = sr.empty8(rows, cols)
    q.view(torch.uint8).copy_(b)
    s.view(torch.uint8).view(-1).copy_(P.order_scales(e, rows, cols))
    return q, s, b.cuda().view(torch.float8_e4m3fn).float().double() * torch.pow(2.0, e.to(F64) - 127).cuda().repeat_interleave(
        128, dim=1)[:, :cols]


def check_product(pc, m, n, k, out, accumulate, ldc=0):  # noqa: F811
    """Every 32 products round once, downwards (2^-23 of the sums' size at most); of fp32 results the sum of a stretch of
    at most 1024 columns does, and the stretches are added to each other."""
    g = P.generator(m + 3 * n + 7 * k)
    qa, sa, a = random8(g, m, k)
    qb, sb, b = random8(g, n, k)
    C = torch.full((m, ldc or n), 7.0, device="cuda").to(TYPES[out])
    c = C[:, :n]
    c0 = 1000 * P.randn(g, m, n).cuda() if accumulate else None
    if accumulate:
        c.copy_(c0)
    sr.precond_gemm8(pc.h, qa, sa, qb, sb, c, accumulate=accumulate)
    sr.precond_gemm8_status(pc.h)
    if ldc:
        assert bool((C[:, n:] == 7.0).all())
    chain = k / 32 + 8 if out == "bf16" else 40 + k / 512
    for r in range(0, m, 1024):
        want, size = a[r:r + 1024] @ b.t(), a[r:r + 1024].abs() @ b.abs().t()
        if accumulate:
            want, size = want + c0[r:r + 1024].double(), size + c0[r:r + 1024].double().abs()
        tol = chain * 2.0 ** -23 * size + (E16 * want.abs() if out == "bf16" else 0)
        bad = (c[r:r + 1024].double() - want).abs() > tol
        assert not bool(bad.any()), (r, int(bad.sum()), bad.nonzero()[:5].tolist())
    # the same bits again, the calls one right after the other
    if not accumulate:
        others = [torch.empty_like(C)[:, :n] for _ in range(2)]
        for o in others:
            sr.precond_gemm8(pc.h, qa, sa, qb, sb, o)
        assert all(torch.equal(o, c) for o in others)


@pytest.mark.parametrize("m,n,k,out,accumulate,ldc", [
    (5000, 4400, 700, "bf16", False, 0),       # pairs, 360 tiles on 76 of them, 6 blocks of K (5 stages), 2 scale groups; whole sectors
    (5000, 4404, 1537, "bf16", False, 0),      # pairs, 13 blocks, 4 groups; 4 elements at a time
    (3000, 3001, 2600, "bf16", False, 0),      # pairs, 144 tiles, 21 blocks; single elements
    (2048, 2048, 4099, "bf16", False, 2064),   # pairs, one tile each, 33 blocks, 9 groups
    (5000, 4400, 700, "f32", False, 0),        # pairs in fp32, one stretch
    (5000, 4404, 1600, "f32", False, 0),       # pairs in fp32, 13 blocks: two stretches a tile, the last of 5 blocks
    (5001, 4403, 1537, "f32", True, 0),        # pairs, accumulating, single elements
    (4096, 1024, 8191, "f32", True, 0),        # pairs, accumulating, 64 blocks, 4 elements at a time
    (5000, 4404, 2048, "f32", True, 4420),     # pairs, accumulating, a pitch
    (5000, 4400, 640, "f32", True, 0),         # single blocks of 128 x 128, 1400 tiles on 152 SMs, accumulating
    (6734, 832, 468, "f32", True, 0),          # single, 371 tiles
    (4000, 2000, 100, "bf16", False, 0),       # pairs, 128 tiles of one block of K each
    (128, 20000, 600, "f32", False, 0),        # one row of tiles
])
def test_products_of_many_tiles(pc, m, n, k, out, accumulate, ldc):  # noqa: F811
    check_product(pc, m, n, k, out, accumulate, ldc)


def test_positive_products_on_pairs(pc):  # noqa: F811
    """A long chain of positive products: the sums of stretches of 1024 columns (32 truncations, of half the final sum on
    average) and 16 additions of them."""
    m, n, k = 2048, 2048, 16384
    x, y = (torch.rand(r, k, generator=P.generator(r + i)) + 0.5 for i, r in enumerate((m, n)))
    (qa, sa), (qb, sb) = sr.empty8(m, k), sr.empty8(n, k)
    sr.precond_quantize8(pc.h, x.cuda(), q=qa, scale=sa)
    sr.precond_quantize8(pc.h, y.cuda(), q=qb, scale=sb)
    c = torch.empty(m, n, device="cuda")
    sr.precond_gemm8(pc.h, qa, sa, qb, sb, c)
    want = sr.dequantize8(qa, sa).double() @ sr.dequantize8(qb, sb).double().t()
    assert float(((c.double() - want) / want).abs().max()) <= (32 + 8 + 16) * 2.0 ** -24


# ------------------------------------------------------------------------------------------------ distillation
def check_large(pc, rows, vocab, top, dtype, launches, in_place=False, tau=2.0):  # noqa: F811
    """On the GPU, some rows at a time.  E32 (4 spread + 32): an exponent's relative error and those of sums and
    exponentials; three times that for the gradient, of q, or where a candidate's q - p cancels of both."""
    g = torch.Generator(device="cuda").manual_seed(rows + vocab)
    z = (3 * torch.randn(rows, vocab, generator=g, device="cuda")).to(TYPES[dtype])
    ids = torch.randint(0, vocab, (rows, top), generator=g, device="cuda", dtype=torch.int32)
    ids[torch.rand(rows, top, generator=g, device="cuda") < 0.2] = -1
    ids[3::7, top // 2:] = ids[3::7, :top - top // 2].clone()          # every id twice
    ids[5::9] = -1                                                     # no candidate
    t = 3 * torch.randn(rows, top, generator=g, device="cuda")
    w = torch.rand(rows, generator=g, device="cuda")
    w[::4] = 0
    z0 = z.clone()
    loss = torch.full((rows,), math.nan, device="cuda")
    grad = z if in_place else torch.full_like(z, math.nan)
    n = sr.precond_launch_count(pc.h)
    sr.precond_distill(pc.h, z, ids, t, loss, weight=w, temperature=tau, dlogits=grad)
    assert sr.precond_launch_count(pc.h) - n == launches
    for r in range(0, rows, 64):
        zr, ir, wr = z0[r:r + 64].double() / tau, ids[r:r + 64].long(), w[r:r + 64].double()
        live = ir >= 0
        tr = torch.where(live, t[r:r + 64].double() / tau, torch.full((), -math.inf, dtype=F64, device="cuda"))
        any_ = live.any(dim=1) & (wr != 0)
        tm = torch.where(any_, tr.amax(dim=1), torch.zeros_like(wr))[:, None]
        p = torch.exp(tr - tm)
        logp = tr - tm - torch.log(p.sum(dim=1, keepdim=True))
        p = torch.where(live, torch.exp(logp), torch.zeros_like(p))
        zm = zr.amax(dim=1, keepdim=True)
        q = torch.exp(zr - zm)
        logs = torch.log(q.sum(dim=1, keepdim=True))
        q = torch.exp(zr - zm - logs)
        logq = zr.gather(1, ir.clamp(min=0)) - zm - logs
        kl = torch.where(live, p * (logp - logq), torch.zeros_like(p)).sum(dim=1)
        want_loss = torch.where(any_, wr * tau * tau * kl, torch.zeros_like(wr))
        spread = (zm[:, 0] - zr.amin(dim=1)) + torch.where(live, (tm - tr), torch.zeros_like(tr)).amax(dim=1)
        unit = (4 * spread + 32) * E32
        assert bool(((loss[r:r + 64].double() - want_loss).abs() <= wr * tau * tau * unit + 4 * E32 * want_loss.abs()).all())
        cand = torch.zeros_like(q).scatter_add_(1, ir.clamp(min=0), live.double()).clamp(max=1)
        q.scatter_add_(1, ir.clamp(min=0), -p)
        want = torch.where(any_[:, None], q, torch.zeros_like(q)) * (wr * tau)[:, None]
        tol = 3 * unit[:, None] * (want.abs() + cand * (wr * tau)[:, None]) + 1e-30
        if dtype == "bf16":
            tol = tol + E16 * want.abs()
        bad = (grad[r:r + 64].double() - want).abs() > tol
        assert not bool(bad.any()), (r, int(bad.sum()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("rows,vocab,top,dtype,launches", [
    (930, 131071, 50, "bf16", 2),      # 4 blocks a row, 8 vectors a thread, candidates in a kernel of their own; odd rows
    (1000, 131072, 128, "bf16", 2),    # the same, aligned
    (460, 151936, 30, "f32", 2),       # 8 blocks a row, rows read twice, candidates in a kernel of their own
    (460, 262147, 300, "bf16", 2),     # the same in bf16, candidates in shared memory
    (455, 262147, 300, "bf16", 1),     # just too few rows for that: beside the stream
    (5, 151937, 30, "f32", 1),         # rows read twice, candidates beside them
    (7, 300001, 129, "bf16", 1),
    (950, 40000, 140, "f32", 2),       # 4 blocks a row, candidates in 8 registers a lane
    (1900, 20001, 1024, "bf16", 2),    # one block a row
])
def test_large_vocabularies(pc, rows, vocab, top, dtype, launches):  # noqa: F811
    check_large(pc, rows, vocab, top, dtype, launches)
    check_large(pc, rows, vocab, top, dtype, launches + (launches == 2), in_place=True)


@pytest.mark.parametrize("rows,vocab,launches", [(2200, 120, 2), (990, 33001, 2), (330, 33001, 1)])
def test_masks(pc, rows, vocab, launches):  # noqa: F811
    """Rows without candidates, repeated ids, ids outside the vocabulary, masked logits, zero weights over NaN: where the
    candidates have a kernel of their own (also of rows that 4 blocks share), and in clusters."""
    low = torch.finfo(torch.float32).min
    z, ids, t, w = distill_inputs(rows, vocab, 12, "f32", masked=False)
    ids[0::11] = -1
    t[1::11] = -math.inf
    ids[2::11] = ids[2::11, :1]
    ids[3::11, 0], ids[3::11, 1] = vocab, 2 ** 31 - 1
    z[4::11, vocab // 2:] = -math.inf
    ids[4::11] = torch.arange(12, dtype=torch.int32)
    z[5::11] = low
    z[6::11] = math.nan
    w[6::11] = 0
    z[7::11] = 1e30
    z[8::11, 1:] = low
    ids[8::11] = torch.arange(12, dtype=torch.int32)
    t[8::11, 1:] = -math.inf
    n = sr.precond_launch_count(pc.h)
    a = check_distill(pc, z, ids, t, w, 1.0)
    assert sr.precond_launch_count(pc.h) - n == launches
    check_distill(pc, z, ids, t, w, 0.25)
    b = check_distill(pc, z, ids, t, w, 1.0, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------------------ streams and graphs
def test_workspaces_of_the_allocator_in_graphs_and_on_streams(pc):  # noqa: F811
    """Calls that take their workspace from torch's allocator, and the distillation of several kernels: on a stream of
    their own and inside a CUDA graph, replayed twice, they give what they give on the current stream."""
    g = P.generator(9)
    rows, cols, vocab, top = 2000, 700, 900, 11
    x, dy = (P.randn(g, rows, cols).bfloat16().cuda() for _ in range(2))
    w = P.randn(g, cols).cuda()
    rstd = torch.rand(rows, generator=g).cuda()
    z, ids, t, wt = (a.cuda() for a in distill_inputs(rows, vocab, top, "bf16"))
    assert sr.precond_distill_workspace(rows, vocab, top, torch.bfloat16) > 0

    def outputs():
        e = torch.empty
        return dict(loss=e(rows, device="cuda"), dz=torch.empty_like(z), over=torch.empty_like(z), loss2=e(rows, device="cuda"),
                    dx=torch.empty_like(x), dw=e(cols, device="cuda"))

    def go(o):
        sr.precond_rms_norm_grad(pc.h, dy, x, w, rstd, o["dx"], o["dw"])
        sr.precond_distill(pc.h, z, ids, t, o["loss"], weight=wt, dlogits=o["dz"])
        o["over"].copy_(z)
        sr.precond_distill(pc.h, o["over"], ids, t, o["loss2"], weight=wt, dlogits=o["over"])

    first = outputs()
    go(first)
    torch.cuda.synchronize()
    assert torch.equal(first["loss"], first["loss2"]) and torch.equal(first["dz"], first["over"])
    side, second = torch.cuda.Stream(), outputs()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            go(second)
    side.synchronize()
    third = outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(third)
    for _ in range(2):
        for v in third.values():
            v.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bytes_of(first[k]), bytes_of(third[k])) for k in first)
    assert all(torch.equal(bytes_of(first[k]), bytes_of(second[k])) for k in first)
