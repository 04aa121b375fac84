"""The operators of a policy's training step in 64 bits on the CPU, straight from their formulas (no code shared with
the library)."""
import math

import torch

F64 = torch.float64


def layer_norm(x, r, w, b, eps):
    """(h, y, mean, rstd); h rounded to x's type, the rest in 64 bits."""
    h = x if r is None else (x.to(F64) + r.to(F64)).to(torch.float32).to(x.dtype)
    f = h.to(F64)
    mean = f.mean(dim=1)
    rstd = 1 / torch.sqrt(((f - mean[:, None]) ** 2).mean(dim=1) + eps)
    y = (f - mean[:, None]) * rstd[:, None] * w.to(F64) + (0 if b is None else b.to(F64))
    return h, y, mean, rstd


def layer_norm_grad(dy, x, w, mean, rstd, dr):
    dy, x, w, m, r = dy.to(F64), x.to(F64), w.to(F64), mean.to(F64)[:, None], rstd.to(F64)[:, None]
    n, g = (x - m) * r, dy * w
    dx = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
    return dx if dr is None else dx + dr.to(F64), (dy * n).sum(dim=0), dy.sum(dim=0)


def policy(z, ids, adv, old, ref, weight, tau, low, high, kl):
    """(loss, logp, dlogits) in 64 bits, one row at a time; adv None: logp alone."""
    rows, vocab = z.shape
    loss, logp, grad = torch.zeros(rows, dtype=F64), torch.zeros(rows, dtype=F64), torch.zeros(rows, vocab, dtype=F64)
    for i in range(rows):
        w, id_ = 1.0 if weight is None else float(weight[i]), int(ids[i])
        if w == 0 or not 0 <= id_ < vocab:
            continue
        logq = torch.log_softmax(z[i].to(F64) / tau, dim=0)
        s = float(logq[id_])
        logp[i] = s
        if adv is None:
            continue
        a = float(adv[i])
        ratio = 1.0 if old is None else math.exp(s - float(old[i]))
        held = min(max(ratio, 1 - low), 1 + high)
        if ratio * a > held * a:
            value, slope = -held * a, 0.0
        else:
            value, slope = -ratio * a, -ratio * a
        if kl and ref is not None:
            d = float(ref[i]) - s
            value += kl * (math.expm1(d) - d)
            slope += -kl * math.expm1(d)
        loss[i] = w * value
        # 1 - q of the taken token as the sum of the others
        others = torch.logsumexp(torch.cat([logq[:id_], logq[id_ + 1:], torch.full((1,), -math.inf, dtype=F64)]), dim=0)
        g = -logq.exp()
        g[id_] = torch.exp(others)
        grad[i] = w * slope / tau * g
    return loss, logp, grad


def grad_norm(tensors):
    return math.sqrt(math.fsum(float((t.to(F64) ** 2).sum()) for t in tensors))
