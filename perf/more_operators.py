"""Cases of the operators that train a policy around the preconditioner: their plain forms and the library's.

* ``norm``       h = x + r, y = (h - mean) / std * w + b: layer norm, y kept or rounded to 8 bits in blocks of 128 columns
* ``norm_grad``  its gradients: dx (with the residual branch's gradient added), dw and db
* ``policy``     the clipped policy loss of taken tokens with a KL term against a reference, and the gradient of the logits
* ``score``      the log probabilities of taken tokens (an old or a reference policy's)
* ``clip``       the norm of a list of gradients, and the gradients scaled down to a largest norm, in place
* ``total``      that norm alone

8-bit values are float8_e4m3fn and scales float8_e8m0fnu, both returned as they are: tensors of these types hold
the values themselves.  Scales lie in the order [512-column group][128-row block][row % 32][row // 32 % 4][block of
128 in the group]; rows and blocks past the end hold 1.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
GROUP = 512
EPS = 1e-5
LOW, HIGH, KL = 0.2, 0.28, 0.04
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decoder with d = 1024 (latency only)
        {"name": "norm-1x1024", "op": "norm", "rows": 1, "cols": 1024, "dtype": "bf16", "residual": True, "out": "q"},
        # a batch of sequences in front of a 6144-wide product in 8 bits
        {"name": "norm-8192x6144", "op": "norm", "rows": 8192, "cols": 6144, "dtype": "bf16", "residual": True, "out": "q"},
        # a ragged microbatch, fp32 stream of a small model
        {"name": "norm_grad-777x1000-f32", "op": "norm_grad", "rows": 777, "cols": 1000, "dtype": "f32", "residual": False},
        # the backward pass of a large batch, the residual branch's gradient joined in
        {"name": "norm_grad-16384x4096", "op": "norm_grad", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True},
        # a few answers scored under the reference policy; odd vocabulary
        {"name": "score-24x50001", "op": "score", "rows": 24, "vocab": 50001, "dtype": "bf16", "tau": 1.0},
        # an update of a small policy in fp32, sampled at a temperature
        {"name": "policy-1000x32000-f32", "op": "policy", "rows": 1000, "vocab": 32000, "dtype": "f32", "tau": 0.7, "kl": True},
        # a ragged microbatch over a vocabulary whose rows begin at no multiple of 16 bytes, without a reference policy
        {"name": "policy-2999x50001", "op": "policy", "rows": 2999, "vocab": 50001, "dtype": "bf16", "tau": 1.0, "kl": False},
        # an update over a large vocabulary
        {"name": "policy-8192x131072", "op": "policy", "rows": 8192, "vocab": 131072, "dtype": "bf16", "tau": 1.0, "kl": True},
        # the gradients of one small layer: a weight, its bias and a norm (latency only)
        {"name": "clip-layer-256x128-f32", "op": "clip", "count": 1, "m": 256, "n": 128, "dtype": "f32", "vectors": 2},
        # a small model of many ragged layers, gradients of both types
        {"name": "clip-97-of-500x333", "op": "clip", "count": 97, "m": 500, "n": 333, "dtype": "bf16", "vectors": 3},
        # 24 decoder layers of d = 1024, six times 1024 x 2048 each, with the fp32 gradients of their norms
        {"name": "clip-144-of-1024x2048", "op": "clip", "count": 144, "m": 1024, "n": 2048, "dtype": "bf16", "vectors": 1},
        # four wide layers in fp32, watched and not clipped
        {"name": "total-4-of-6144x6144-f32", "op": "total", "count": 4, "m": 6144, "n": 6144, "dtype": "f32", "vectors": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "policy", "policy", "score", "clip", "clip", "total"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = max(64, cols // 128 * 128)
        case = {"op": op, "rows": _log(rng, 1, min(32768, 50_000_000 // cols)), "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.7}
        return dict(case, out=rng.choice(["q", "y"])) if op == "norm" else case
    if op in ("policy", "score"):
        vocab = _log(rng, 500, 160000)
        case = {"op": op, "rows": _log(rng, 1, min(8192, 500_000_000 // vocab)), "vocab": vocab, "dtype": dtype,
                "tau": rng.choice([0.7, 1.0, 1.0, 1.3])}
        return dict(case, kl=rng.random() < 0.6) if op == "policy" else case
    m, n = _log(rng, 16, 4096), _log(rng, 16, 4096)
    return {"op": op, "count": _log(rng, 1, min(400, max(1, 300_000_000 // (m * n)))), "m": m, "n": n, "dtype": dtype,
            "vectors": rng.randint(0, 3)}


# --------------------------------------------------------------------------------------------- 8-bit form
def _pad_to(n, b):
    return -(-n // b) * b


def _scale_order(e):
    """Exponents [rows padded to 128, blocks padded to 4] in the order the product reads them, as e8m0."""
    R, K = e.shape
    e = (e + 127).to(torch.uint8).view(R // 128, 4, 32, K // 4, 4).permute(3, 0, 2, 1, 4).contiguous()
    return e.view(torch.float8_e8m0fnu)


def _to8(x):
    """float32 x [rows, cols] in 8-bit form: values and scales, one for each row and 128 columns."""
    rows, cols = x.shape
    R, K = _pad_to(rows, 128), _pad_to(cols, GROUP)
    p = torch.zeros(R, K, device=x.device)
    p[:rows, :cols] = x
    b = p.view(R, K // 128, 128)
    amax = b.abs().amax(dim=2, keepdim=True)
    m, k = torch.frexp(amax)
    e = k - 9 + (m > 0.875).to(k.dtype)                # the least e with amax <= 448 2^e: 448 = 0.875 2^9
    e = torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))
    q = (b * ((127 - e) << 23).view(torch.float32)).to(torch.float8_e4m3fn).view(R, K)[:rows, :cols]
    e = e.reshape(R, K // 128).clone()
    e[rows:] = 0
    e[:, -(-cols // 128):] = 0
    return q, _scale_order(e)


def _held8(rows, cols, device):
    """An 8-bit matrix as a program keeps it: rows 16 bytes apart or a multiple of that."""
    return torch.zeros(rows, _pad_to(cols, 16), dtype=torch.float8_e4m3fn, device=device)[:, :cols]


def _scales(rows, cols, device):
    s = torch.zeros(_pad_to(cols, GROUP) // GROUP, _pad_to(rows, 128) // 128, 32, 4, 4, dtype=torch.uint8, device=device)
    return s.view(torch.float8_e8m0fnu)


# --------------------------------------------------------------------------------------------- inputs
def _stream(gen, rows, cols, dev):
    """Activations: columns of different size, a few of them large, and rows with a mean of their own."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    c = torch.exp(0.5 * torch.randn(cols, generator=gen, device=dev))
    c = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.01, 10 * c, c)
    return x * c + torch.randn(rows, 1, generator=gen, device=dev)


def _gradient(gen, rows, cols, dev):
    """Output gradients: rows of very different size (tokens already learnt have small ones)."""
    return torch.randn(rows, cols, generator=gen, device=dev) * torch.exp(2 * torch.randn(rows, 1, generator=gen, device=dev)) * 1e-4


def _sizes(case):
    """The list's shapes and types: weights, and after each the vectors beside it (biases, norms) in fp32."""
    out = []
    for i in range(case["count"]):
        out.append(((case["m"], case["n"]), TYPES[case["dtype"]]))
        out += [((case["m"] if v % 2 else case["n"],), torch.float32) for v in range(case["vectors"])]
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": case}
    if op in ("norm", "norm_grad"):
        rows, cols, dt = case["rows"], case["cols"], TYPES[case["dtype"]]
        st["x"] = _stream(gen, rows, cols, dev).to(dt)
        st["w"] = 1 + 0.2 * torch.randn(cols, generator=gen, device=dev)
        st["mean"], st["rstd"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        if op == "norm":
            st["b"] = 0.2 * torch.randn(cols, generator=gen, device=dev)
            st["r"] = _stream(gen, rows, cols, dev).to(dt) if case["residual"] else None
            st["h"] = torch.empty_like(st["x"]) if case["residual"] else None
            st["y"] = torch.empty_like(st["x"]) if case["out"] == "y" else None
            st["q"], st["s"] = (_held8(rows, cols, dev), _scales(rows, cols, dev)) if case["out"] == "q" else (None, None)
        else:
            st["dy"] = _gradient(gen, rows, cols, dev).to(dt)
            st["dr"] = _gradient(gen, rows, cols, dev).to(dt) if case["residual"] else None
            st["dx"] = torch.empty_like(st["x"])
            st["dw"], st["db"] = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
            x = st["x"].double()                                   # the forward pass left these
            st["mean"] = x.mean(1).float()
            st["rstd"] = torch.rsqrt((x - x.mean(1, keepdim=True)).square_().mean(1) + EPS).float()
        return st
    if op in ("policy", "score"):
        rows, vocab = case["rows"], case["vocab"]
        z = torch.randn(rows, vocab, generator=gen, device=dev).mul_(2.5 * case["tau"])
        # the taken tokens were sampled: the largest z / tau + Gumbel noise
        noise = torch.empty_like(z).exponential_(generator=gen).log_().neg_()
        st["ids"] = noise.add_(z, alpha=1 / case["tau"]).argmax(dim=1)
        del noise
        st["z"] = z.to(TYPES[case["dtype"]])
        st["logp"] = torch.empty(rows, device=dev)
        if op == "policy":
            now = (z.gather(1, st["ids"][:, None])[:, 0] / case["tau"] - torch.logsumexp(z.div_(case["tau"]), dim=1))
            # the policy has moved since the tokens were drawn, and farther from the reference
            st["old"] = now + 0.15 * torch.randn(rows, generator=gen, device=dev)
            st["ref"] = now + 0.3 * torch.randn(rows, generator=gen, device=dev) if case["kl"] else None
            st["adv"] = torch.randn(rows, generator=gen, device=dev)
            # one row in eight is a prompt's or padding: its weight is zero, and so is what is known of it
            live = (torch.rand(rows, generator=gen, device=dev) > 0.125).float()
            st["weight"] = live / live.sum().clamp(min=1)
            st["loss"] = torch.empty(rows, device=dev)
            st["dz"] = torch.empty_like(st["z"])
        return st
    # as data-parallel training keeps them: the gradients are views of one flat buffer for each type
    flat = {}
    for name, dt in TYPES.items():
        n = sum(math.prod(shape) for shape, t in _sizes(case) if t == dt)
        if n:
            flat[name] = torch.empty(n, dtype=dt, device=dev)
    at = dict.fromkeys(flat, 0)
    grads = []
    for shape, dt in _sizes(case):
        name, n = "bf16" if dt == torch.bfloat16 else "f32", math.prod(shape)
        g = flat[name][at[name]:at[name] + n].view(shape)
        at[name] += n
        # layers' gradients differ in size
        g.copy_(torch.randn(*shape, generator=gen, device=dev).mul_(1e-3 * torch.exp(0.7 * torch.randn(1, generator=gen, device=dev))))
        grads.append(g)
    st["grads"], st["flat"], st["norm"] = grads, flat, torch.empty((), device=dev)
    st["limit"] = 0.6 * math.sqrt(sum(float(f.float().square_().sum()) for f in flat.values()))
    if own:
        import shampoo_roots_gb300 as sr
        st["list"] = sr.TensorList(grads)                          # the buffers are a training program's for the whole run
    return st


_kept = []


def _library():
    """The package and the handle that a program keeps for the whole run."""
    if not _kept:
        import shampoo_roots_gb300 as sr
        _kept.append((sr, sr.Preconditioner(torch.cuda.current_device())))
    return _kept[0]


# --------------------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _limit(st):
    """The largest norm of this pass.  It falls a little from pass to pass, so that every pass finds gradients to scale
    down, as every step's new ones are."""
    limit = st["limit"]
    st["limit"] *= 0.999
    return limit


def _run_own(st):
    sr, pc = _library()
    h, op, case = pc.h, st["op"], st["case"]
    if op == "norm":
        sr.precond_layer_norm(h, st["x"], st["w"], EPS, bias=st["b"], residual=st["r"], total=st["h"], y=st["y"], q=st["q"],
                              scale=st["s"], mean=st["mean"], rstd=st["rstd"])
        out = {"mean": st["mean"], "rstd": st["rstd"]}
        out.update({"y": st["y"]} if case["out"] == "y" else {"q": st["q"], "scale": st["s"]})
        return dict(out, h=st["h"]) if case["residual"] else out
    if op == "norm_grad":
        sr.precond_layer_norm_grad(h, st["dy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], db=st["db"],
                                   dresidual=st["dr"])
        return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}
    if op == "score":
        sr.precond_policy(h, st["z"], st["ids"], temperature=case["tau"], logp=st["logp"])
        return st["logp"]
    if op == "policy":
        sr.precond_policy(h, st["z"], st["ids"], advantage=st["adv"], old_logp=st["old"], ref_logp=st["ref"], weight=st["weight"],
                          temperature=case["tau"], clip_low=LOW, clip_high=HIGH, kl=KL if case["kl"] else 0.0, loss=st["loss"],
                          logp=st["logp"], dlogits=st["dz"])
        return {"loss": st["loss"], "logp": st["logp"], "dlogits": st["dz"]}
    if op == "clip":
        sr.precond_clip_grads(h, st["list"], _limit(st), st["norm"])
        return {"norm": st["norm"], "grads": st["flat"]}
    sr.precond_grad_norm(h, st["list"], st["norm"])
    return st["norm"]


def _run_plain(st):
    op, case = st["op"], st["case"]
    if op == "norm":
        h = st["x"]
        if case["residual"]:
            h = (h.float() + st["r"].float()).to(h.dtype)          # the stream keeps its type
        f = h.float()
        mean = f.mean(dim=1)
        d = f - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(dim=1) + EPS)
        y = d * rstd[:, None] * st["w"] + st["b"]
        out = {"mean": mean, "rstd": rstd}
        if case["out"] == "y":
            out["y"] = y.to(h.dtype)
        else:
            out["q"], out["scale"] = _to8(y)
        return dict(out, h=h) if case["residual"] else out
    if op == "norm_grad":
        dy, r = st["dy"].float(), st["rstd"][:, None]
        n = (st["x"].float() - st["mean"][:, None]) * r
        g = dy * st["w"]
        dx = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
        if case["residual"]:
            dx = dx + st["dr"].float()
        return {"dx": dx.to(st["dy"].dtype), "dw": (dy * n).sum(dim=0), "db": dy.sum(dim=0)}
    if op in ("policy", "score"):
        z = st["z"].float() / case["tau"]
        m = z.amax(dim=1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(dim=1, keepdim=True)
        logp = (z.gather(1, st["ids"][:, None]) - m - torch.log(total))[:, 0]
        if op == "score":
            return logp
        w, a = st["weight"], st["adv"]
        logp = torch.where(w != 0, logp, torch.zeros_like(logp))   # rows of weight zero are left out
        ratio = torch.exp(logp - st["old"])
        free, held = ratio * a, ratio.clamp(1 - LOW, 1 + HIGH) * a
        loss = -torch.minimum(free, held)
        slope = torch.where(free <= held, -free, torch.zeros_like(free))
        if case["kl"]:
            d = st["ref"] - logp
            loss = loss + KL * (torch.exp(d) - d - 1)
            slope = slope + KL * (1 - torch.exp(d))
        loss, slope = loss * w, slope * w / case["tau"]
        e.div_(total).mul_(-slope[:, None])
        e.scatter_add_(1, st["ids"][:, None], slope[:, None])
        return {"loss": loss, "logp": logp, "dlogits": e.to(st["z"].dtype)}
    total = torch.zeros((), device="cuda")
    for g in st["grads"]:
        f = g.float()
        total = total + (f * f).sum()
    norm = total.sqrt()
    if op == "total":
        return norm
    c = (_limit(st) / norm).clamp(max=1.0)
    for g in st["grads"]:
        g.copy_(g.float() * c)
    return {"norm": norm, "grads": st["flat"]}


# --------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols, b = case["rows"], case["cols"], SIZE[case["dtype"]]
        n = rows * cols
        if op == "norm":
            out = b if case["out"] == "y" else 1 + 1 / 128
            return {"bytes": n * (b * (3 if case["residual"] else 1) + out) + 8 * rows + 8 * cols, "flops": 10 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + 8 * rows + 12 * cols, "flops": 13 * n}
    if op in ("policy", "score"):
        n, b = case["rows"] * case["vocab"], SIZE[case["dtype"]]
        if op == "score":
            return {"bytes": n * b + 12 * case["rows"], "flops": 4 * n}
        # rows of weight zero (one in eight) need no reading, and a zero gradient written
        return {"bytes": n * b * 1.875 + 36 * case["rows"], "flops": 6 * n}
    n = sum(math.prod(shape) for shape, _ in _sizes(case))
    b = sum(math.prod(shape) * (2 if dt == torch.bfloat16 else 4) for shape, dt in _sizes(case))
    return {"bytes": b * (2 if op == "clip" else 1) + 4, "flops": n * (3 if op == "clip" else 2)}


# --------------------------------------------------------------------------------------------- 64 bits
def _before8(x):
    """What an 8-bit matrix stands for, before its rounding: x over its block's scale.  (A value in the middle of two
    8-bit numbers goes either way with its last fp32 bit, so that the rounded ones say little.)"""
    rows, cols = x.shape
    blocks = -(-cols // 128)
    p = torch.nn.functional.pad(x, (0, blocks * 128 - cols)).view(rows, blocks, 128)
    amax = p.abs().amax(dim=2)
    two_to = lambda k: ((k.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / E4M3_MAX))
    e = torch.where(amax > E4M3_MAX * two_to(e), e + 1, torch.where(amax <= E4M3_MAX * two_to(e - 1), e - 1, e))
    e = torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))
    return (p / two_to(e)[:, :, None]).reshape(rows, blocks * 128)[:, :cols]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        h = st["x"]
        out = {}
        if case["residual"]:
            h = (h.double() + st["r"].double()).to(h.dtype)        # h as the stream holds it
            out["h"] = h.double()
        x = h.double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        std = torch.sqrt(var + EPS)
        y = torch.addcmul(st["b"].double(), (x - mean[:, None]) / std[:, None], st["w"].double())
        out["mean"], out["rstd"] = mean, 1 / std
        # a block whose largest value is at the boundary of two scales goes with its last bit: no scale is given
        out.update({"y": y} if case["out"] == "y" else {"q": _before8(y), "scale": None})
        return out
    if op == "norm_grad":
        x, dy, w, r = st["x"].double(), st["dy"].double(), st["w"].double(), st["rstd"].double()
        c = x - st["mean"].double()[:, None]
        dot = torch.einsum("tc,c,tc->t", dy, w, c)
        flat = torch.einsum("tc,c->t", dy, w)
        dx = dy * w * r[:, None] - (r * flat / case["cols"])[:, None] - c * (r ** 3 * dot / case["cols"])[:, None]
        if case["residual"]:
            dx = dx + st["dr"].double()
        return {"dx": dx, "dw": torch.einsum("tc,tc,t->c", dy, c, r), "db": dy.sum(dim=0)}
    if op in ("policy", "score"):
        losses, logps, grads = [], [], []
        for a in range(0, case["rows"], 512):                      # a few rows at a time: 64 bits of a large vocabulary
            part = slice(a, a + 512)
            ids = st["ids"][part, None]
            logq = torch.log_softmax(st["z"][part].double() / case["tau"], dim=1)
            s = logq.gather(1, ids)[:, 0]
            if op == "score":
                logps.append(s)
                continue
            w, adv = st["weight"][part].double(), st["adv"][part].double()
            s = torch.where(w != 0, s, torch.zeros_like(s))
            ratio = torch.exp(s - st["old"][part].double())
            clipped = ((adv > 0) & (ratio > 1 + HIGH)) | ((adv < 0) & (ratio < 1 - LOW))
            loss = -adv * torch.where(clipped, torch.where(adv > 0, 1 + HIGH, 1 - LOW), ratio)
            slope = torch.where(clipped, torch.zeros_like(adv), -adv * ratio)
            if case["kl"]:
                x = st["ref"][part].double() - s
                loss = loss + KL * (torch.expm1(x) - x)
                slope = slope - KL * torch.expm1(x)
            losses.append(w * loss)
            logps.append(s)
            g = logq.exp_().neg_()
            g.scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.float64))
            grads.append((g * (w * slope / case["tau"])[:, None]).to(torch.float32 if case["rows"] * case["vocab"] > 1e8 else torch.float64))
        if op == "score":
            return torch.cat(logps)
        return {"loss": torch.cat(losses), "logp": torch.cat(logps), "dlogits": torch.cat(grads)}
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in st["grads"]))
    out = torch.tensor(norm, dtype=torch.float64, device="cuda")
    if op == "total":
        return out
    c = min(1.0, st["limit"] / norm)
    return {"norm": out, "grads": {name: f.double() * c for name, f in st["flat"].items()}}
