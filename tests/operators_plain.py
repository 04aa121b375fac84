"""The training-step operators in 64 bits on the CPU, straight from their formulas (no code shared with the
library), and inputs for them."""
import math

import torch

F64 = torch.float64


def blocks(cols):
    return -(-cols // 128)


def order_scales(exps, rows, cols):
    """Biased exponents [rows, blocks] in the library's order: index arithmetic, one byte at a time."""
    G, R = -(-cols // 512), -(-rows // 128)
    out = torch.full((G * R * 512,), 127, dtype=torch.uint8)
    r = torch.arange(rows)[:, None]
    k = torch.arange(blocks(cols))[None, :]
    at = ((k // 4) * R + r // 128) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    out[at.reshape(-1)] = exps.to(torch.uint8).reshape(-1)
    return out


def exponents(amax):
    """Least e >= -127 with amax <= 448 2^e (0 for an empty block), 64 bits."""
    e = torch.zeros(amax.shape, dtype=torch.int64)
    if amax.numel() == 0:
        return e
    flat = [0 if a == 0 else max(-127, math.frexp(a)[1] - 9 + (math.frexp(a)[0] > 0.875)) for a in amax.reshape(-1).tolist()]
    e.view(-1).copy_(torch.tensor(flat, dtype=torch.int64))
    return e


def quantize(x, tile=False):
    """(e4m3 values as float64, biased exponents [rows, blocks]) of a matrix whose values are fp32 numbers."""
    x = x.to(F64)
    rows, cols = x.shape
    p = torch.zeros(rows, blocks(cols) * 128, dtype=F64)
    p[:, :cols] = x
    b = p.view(rows, blocks(cols), 128)
    fin = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b))
    amax = fin.amax(dim=2)
    if tile:
        amax = amax.clone()
        for r in range(0, rows, 128):
            amax[r:r + 128] = amax[r:r + 128].amax(dim=0, keepdim=True)
    e = exponents(amax)
    y = torch.where(torch.isfinite(b), b * torch.pow(2.0, -e.to(F64))[:, :, None], torch.full_like(b, math.nan))
    # x 2^-e is exact in fp32, and the cast rounds to nearest even
    q = y.to(torch.float32).to(torch.float8_e4m3fn).to(F64).view(rows, blocks(cols) * 128)[:, :cols]
    return q, e + 127


def dequantize(q, exps):
    cols = q.shape[1]
    v = torch.pow(2.0, exps.to(F64) - 127).repeat_interleave(128, dim=1)[:, :cols]
    return q.to(F64) * v


def rms_norm(x, r, w, eps):
    """(h, y, rstd); h rounded to x's type, the rest in 64 bits."""
    h = x if r is None else (x.to(F64) + r.to(F64)).to(torch.float32).to(x.dtype)
    f = h.to(F64)
    rstd = 1 / torch.sqrt((f * f).mean(dim=1) + eps)
    return h, f * rstd[:, None] * w.to(F64), rstd


def rms_norm_grad(dy, x, w, rstd, dr):
    dy, x, w, r = dy.to(F64), x.to(F64), w.to(F64), rstd.to(F64)[:, None]
    n, g = x * r, dy * w
    dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
    return dx if dr is None else dx + dr.to(F64), (dy * n).sum(dim=0)


def distill(z, ids, t, weight, tau):
    """(loss, dlogits) in 64 bits, one row at a time."""
    rows, vocab = z.shape
    loss, grad = torch.zeros(rows, dtype=F64), torch.zeros(rows, vocab, dtype=F64)
    for i in range(rows):
        w = 1.0 if weight is None else float(weight[i])
        ok = (ids[i] >= 0) & (ids[i] < vocab) & (t[i].to(F64) != -math.inf)
        if w == 0 or not bool(ok.any()):
            continue
        id_, ti = ids[i][ok].long(), t[i][ok].to(F64) / tau
        logq = torch.log_softmax(z[i].to(F64) / tau, dim=0)
        logp = torch.log_softmax(ti, dim=0)
        p = logp.exp()
        loss[i] = w * tau * tau * (p * (logp - logq[id_])).sum()
        g = logq.exp()
        g.index_add_(0, id_, -p)
        grad[i] = w * tau * g
    return loss, grad


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen)


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def pitched(x, pitch, device="cuda", offset=0):
    """x on the device with rows `pitch` elements apart, starting `offset` elements into its buffer; what lies
    between the rows is NaN."""
    rows, cols = x.shape
    buf = torch.full((rows * pitch + offset + 64,), math.nan, dtype=torch.float32).to(x.dtype).to(device)
    v = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(x)
    return v
