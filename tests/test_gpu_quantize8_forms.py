"""precond_quantize8 of a matrix that is in 8-bit form already: what its values are in fp32 decides, so that a value
beyond fp32's range and every value under the scale byte 255 become NaN and count for no block's largest."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
from test_gpu_operators import pc, same8  # noqa: F401  (pc: the handle's fixture)

pytestmark = pytest.mark.gpu


def again(pc, q, s, tile):  # noqa: F811
    """The form put into 8 bits again, both ways at once and each alone, against the plain form of its fp32 values."""
    rows, cols = q.shape
    v = sr.dequantize8(q.cpu(), s.cpu())
    block = sr.BLOCK_TILE if tile else sr.BLOCK_ROW
    for ways in ("both", "rows", "columns"):
        o, os_ = sr.empty8(rows, cols) if ways != "columns" else (None, None)
        ot, ots = sr.empty8(cols, rows) if ways != "rows" else (None, None)
        sr.precond_quantize8(pc.h, q, x_scale=s, q=o, scale=os_, qt=ot, scale_t=ots, block=block)
        if o is not None:
            same8(o, os_, *P.quantize(v, tile), ways + ": rows")
        if ot is not None:
            same8(ot, ots, *P.quantize(v.t().contiguous(), tile), ways + ": columns")
    return v


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_that_round_beyond_fp32(pc, tile, dtype):  # noqa: F811
    """3.4e38 is 256 x 2^120 in 8-bit form, which fp32 does not hold."""
    x = P.randn(P.generator(3), 200, 300).to(dtype)
    big = torch.finfo(dtype).max
    x[0, 0], x[5, 130], x[40, 299], x[199, 7] = big, -big, big / 1.02, -big / 2
    x[60] = 0
    x[60, 200] = -big                                  # the only value of its block
    q, s = sr.empty8(200, 300)
    sr.precond_quantize8(pc.h, x.cuda(), q=q, scale=s)
    v = again(pc, q, s, tile)
    assert int((~v.isfinite()).sum()) == 4 and bool(v[199, 7].isfinite())


@pytest.mark.parametrize("tile", [False, True])
def test_scale_bytes_at_the_ends(pc, tile):  # noqa: F811
    """255 is no scale: all of its block is NaN, zeros too.  254 and 0 are 2^127 and 2^-127."""
    g = P.generator(4)
    e4m3 = torch.randint(0, 256, (140, 520), generator=g, dtype=torch.uint8)
    e4m3[(e4m3 & 127) == 127] = 0                      # no NaN among the values, but for the rows below
    exps = torch.randint(100, 150, (140, 5), generator=g)
    exps[3, 1], exps[20, 0], exps[139, 4], exps[70] = 255, 255, 255, 255
    e4m3[20, :128] = 0
    exps[30, 2], exps[31, 2], exps[32] = 254, 0, 247
    e4m3[30, 256:300] = 0x38                           # 1: 2^127 is a number, the larger ones are not
    e4m3[50, 17] = 0x7F
    q, s = sr.empty8(140, 520)
    q.view(torch.uint8).copy_(e4m3)
    s.view(torch.uint8).view(-1).copy_(P.order_scales(exps, 140, 520))
    v = again(pc, q, s, tile)
    assert bool(v[3, 128:256].isnan().all()) and bool(v[20, :128].isnan().all()) and bool(v[70].isnan().all())
    assert bool(v[30, 256:300].isfinite().all()) and math.isnan(v[50, 17])
