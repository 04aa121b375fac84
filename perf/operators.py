"""Cases of the training-step operators around the preconditioner: their plain forms and the library's.

The operators are those of an 8-bit weight matrix's training step, whose last result is the gradient that the
preconditioner takes:

* ``norm``      h = x + r, y = h / rms(h) * w, y rounded to 8 bits in blocks of 128 columns
* ``norm_grad`` the gradients of that norm: dx (with the residual branch's gradient added) and dw
* ``quantize``  a matrix rounded to 8 bits, along its rows and along its columns (transposed), with power-of-two scales
* ``gemm``      C = A B^T of two 8-bit matrices with a scale for every row and block of 128 along the contraction
* ``distill``   a student's distillation loss against a teacher's top logits, and the gradient of the logits

8-bit values are float8_e4m3fn and scales float8_e8m0fnu, both returned as they are: tensors of these types hold
the values themselves.  Scales lie in the order [512-column group][128-row block][row % 32][row // 32 % 4][block of
128 in the group]; rows and blocks past the end hold 1.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK, GROUP = 128, 512
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a decoder with d = 1024 (latency only)
        {"name": "norm-1x1024", "op": "norm", "rows": 1, "cols": 1024, "dtype": "bf16", "residual": True},
        # a batch of sequences in front of a 6144-wide product
        {"name": "norm-8192x6144", "op": "norm", "rows": 8192, "cols": 6144, "dtype": "bf16", "residual": True},
        # a ragged microbatch, fp32 stream of a small model
        {"name": "norm_grad-777x1000-f32", "op": "norm_grad", "rows": 777, "cols": 1000, "dtype": "f32", "residual": False},
        # the backward pass of a large batch, the residual branch's gradient joined in
        {"name": "norm_grad-16384x4096", "op": "norm_grad", "rows": 16384, "cols": 4096, "dtype": "bf16", "residual": True},
        # an MLP weight after an optimizer step: 128 x 128 blocks, both orientations
        {"name": "quantize-weight-4096x1024", "op": "quantize", "rows": 4096, "cols": 1024, "dtype": "f32", "block": "tile", "ways": "both"},
        # an output gradient of a ragged batch: by rows for dgrad, by columns for wgrad
        {"name": "quantize-10007x6144", "op": "quantize", "rows": 10007, "cols": 6144, "dtype": "bf16", "block": "row", "ways": "both"},
        # one token through a 6144 x 6144 weight (bound by the weight's bytes)
        {"name": "gemm-1x6144x6144", "op": "gemm", "m": 1, "n": 6144, "k": 6144, "out": "bf16", "accumulate": False},
        # a weight gradient of the 24-layer stack's MLP, accumulated in fp32 over a ragged batch of tokens
        {"name": "gemm-wgrad-4096x1024x8191", "op": "gemm", "m": 4096, "n": 1024, "k": 8191, "out": "f32", "accumulate": True},
        # a large batch through a wide layer
        {"name": "gemm-16384x6144x6144", "op": "gemm", "m": 16384, "n": 6144, "k": 6144, "out": "bf16", "accumulate": False},
        # a few answers scored against a teacher without a backward pass; odd vocabulary
        {"name": "distill-eval-24x50001", "op": "distill", "rows": 24, "vocab": 50001, "top": 20, "dtype": "bf16", "grad": False, "tau": 1.0},
        # a training step of a small student in fp32
        {"name": "distill-1000x32000-f32", "op": "distill", "rows": 1000, "vocab": 32000, "top": 64, "dtype": "f32", "grad": True, "tau": 2.0},
        # a training step over a large vocabulary
        {"name": "distill-8192x131072", "op": "distill", "rows": 8192, "vocab": 131072, "top": 128, "dtype": "bf16", "grad": True, "tau": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "gemm", "gemm", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = max(64, cols // 128 * 128)
        return {"op": op, "rows": _log(rng, 1, min(32768, 50_000_000 // cols)), "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.7}
    if op == "quantize":
        cols = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            cols = max(16, cols // 16 * 16)
        return {"op": op, "rows": _log(rng, 1, min(32768, 60_000_000 // cols)), "cols": cols, "dtype": dtype,
                "block": rng.choice(["row", "tile"]), "ways": rng.choice(["both", "both", "rows", "columns"])}
    if op == "gemm":
        m, n, k = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            n = max(64, n // 64 * 64)
        if rng.random() < 0.5:
            k = max(64, k // 64 * 64)
        k = max(64, min(k, int(3e11 / (m * n))))
        out = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "m": m, "n": n, "k": k, "out": out, "accumulate": out == "f32" and rng.random() < 0.7}
    vocab = _log(rng, 500, 160000)
    return {"op": "distill", "rows": _log(rng, 1, min(8192, 500_000_000 // vocab)), "vocab": vocab,
            "top": _log(rng, 1, 256), "dtype": dtype, "grad": rng.random() < 0.75, "tau": rng.choice([0.5, 1.0, 2.0, 4.0])}


# --------------------------------------------------------------------------------------------- 8-bit form
def _pad_to(n, b):
    return -(-n // b) * b


def _scale_order(e):
    """Exponents [rows padded to 128, blocks padded to 4] in the order the product reads them, as e8m0."""
    R, K = e.shape
    e = (e + 127).to(torch.uint8).view(R // 128, 4, 32, K // 4, 4).permute(3, 0, 2, 1, 4).contiguous()
    return e.view(torch.float8_e8m0fnu)


def _row_exponents(s, rows, blocks):
    """The inverse: float32 scales [rows, blocks]."""
    G, R = s.shape[:2]
    return s.view(torch.uint8).permute(1, 3, 2, 0, 4).reshape(R * 128, G * 4)[:rows, :blocks].contiguous().view(
        torch.float8_e8m0fnu).float()


def _exponents(amax):
    """The least e with amax <= 448 2^e (0 for an empty block), at least -127."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)                # 448 = 0.875 2^9
    return torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))


def _to8(x, block):
    """float32 x [rows, cols] in 8-bit form: values and scales."""
    rows, cols = x.shape
    R, K = _pad_to(rows, 128), _pad_to(cols, GROUP)
    p = torch.zeros(R, K, device=x.device)
    p[:rows, :cols] = x
    b = p.view(R // 128, 128, K // 128, 128)
    amax = b.abs().amax(dim=3, keepdim=True)
    if block == "tile":
        amax = amax.amax(dim=1, keepdim=True).expand(-1, 128, -1, -1)
    e = _exponents(amax)
    back = ((127 - e) << 23).view(torch.float32)        # 2^-e
    q = (b * back).to(torch.float8_e4m3fn).view(R, K)[:rows, :cols]
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


def _from8(q, s):
    """float32 values of an 8-bit matrix."""
    rows, cols = q.shape
    blocks = -(-cols // 128)
    return q.float() * _row_exponents(s, rows, blocks).repeat_interleave(128, dim=1)[:, :cols]


# --------------------------------------------------------------------------------------------- inputs
def _stream(gen, rows, cols, dev):
    """Activations: columns of different size, a few of them large, as a trained network's stream has."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    c = torch.exp(0.5 * torch.randn(cols, generator=gen, device=dev))
    c = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.01, 10 * c, c)
    return x * c


def _gradient(gen, rows, cols, dev):
    """Output gradients: rows of very different size (tokens already learnt have small ones)."""
    return torch.randn(rows, cols, generator=gen, device=dev) * torch.exp(2 * torch.randn(rows, 1, generator=gen, device=dev)) * 1e-4


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = {"op": case["op"], "case": case}
    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols, dt = case["rows"], case["cols"], TYPES[case["dtype"]]
        st["x"] = _stream(gen, rows, cols, dev).to(dt)
        st["w"] = 1 + 0.2 * torch.randn(cols, generator=gen, device=dev)
        st["rstd"] = torch.empty(rows, device=dev)
        if op == "norm":
            st["r"] = _stream(gen, rows, cols, dev).to(dt) if case["residual"] else None
            st["h"] = torch.empty_like(st["x"]) if case["residual"] else None
            st["q"], st["s"] = _held8(rows, cols, dev), _scales(rows, cols, dev)
        else:
            st["dy"] = _gradient(gen, rows, cols, dev).to(dt)
            st["dr"] = _gradient(gen, rows, cols, dev).to(dt) if case["residual"] else None
            st["dx"], st["dw"] = torch.empty_like(st["x"]), torch.empty(cols, device=dev)
            st["rstd"] = torch.rsqrt(st["x"].double().square().mean(1) + EPS).float()    # the forward pass left it
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = 0.02 * torch.randn(rows, cols, generator=gen, device=dev) if case["block"] == "tile" else _gradient(gen, rows, cols, dev)
        st["x"] = x.to(TYPES[case["dtype"]])
        by_rows, by_cols = case["ways"] != "columns", case["ways"] != "rows"
        st["q"], st["s"] = (_held8(rows, cols, dev), _scales(rows, cols, dev)) if by_rows else (None, None)
        st["qt"], st["st"] = (_held8(cols, rows, dev), _scales(cols, rows, dev)) if by_cols else (None, None)
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        wgrad = case["accumulate"]
        a = _gradient(gen, k, m, dev).t() if wgrad else _stream(gen, m, k, dev)
        b = _stream(gen, k, n, dev).t() if wgrad else 0.02 * torch.randn(n, k, generator=gen, device=dev)
        for key, x, block in (("a", a, "row"), ("b", b, "row" if wgrad else "tile")):
            q, s = _to8(x, block)
            st[key] = _held8(q.shape[0], q.shape[1], dev)
            st[key].copy_(q)
            st[key + "s"] = s
            del q, x
        # an accumulated gradient holds the earlier microbatches' sum, and every pass adds to it
        st["out"] = (1e-3 * torch.randn(m, n, generator=gen, device=dev) if wgrad
                     else torch.empty(m, n, dtype=TYPES[case["out"]], device=dev))
    else:
        rows, vocab, top, dt = case["rows"], case["vocab"], case["top"], TYPES[case["dtype"]]
        z = torch.randn(rows, vocab, generator=gen, device=dev)
        t = z + 0.7 * torch.randn(rows, vocab, generator=gen, device=dev)                # the teacher: near the student
        z = z.mul_(2.5).to(dt)
        st["z"] = z
        top = min(top, vocab)
        t, ids = torch.topk(t, top, dim=1)
        st["t"] = 2.5 * t
        del t
        # rows with fewer than `top` candidates are filled up with -1
        keep = torch.randint(max(1, top // 2), top + 1, (rows, 1), generator=gen, device=dev)
        st["ids"] = torch.where(torch.arange(top, device=dev) < keep, ids, torch.full_like(ids, -1))
        # one row in eight is a prompt's or padding: its weight is zero
        w = (torch.rand(rows, generator=gen, device=dev) > 0.125).float()
        st["weight"] = w / w.sum().clamp(min=1)
        st["loss"] = torch.empty(rows, device=dev)
        st["dz"] = torch.empty_like(z) if case["grad"] else None
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


def _run_own(st):
    sr, pc = _library()
    h, op, case = pc.h, st["op"], st["case"]
    if op == "norm":
        sr.precond_rms_norm(h, st["x"], st["w"], EPS, residual=st["r"], total=st["h"], q=st["q"], scale=st["s"],
                            rstd=st["rstd"])
        out = {"q": st["q"], "scale": st["s"], "rstd": st["rstd"]}
        return dict(out, h=st["h"]) if case["residual"] else out
    if op == "norm_grad":
        sr.precond_rms_norm_grad(h, st["dy"], st["x"], st["w"], st["rstd"], st["dx"], st["dw"],
                                 dresidual=st["dr"])
        return {"dx": st["dx"], "dw": st["dw"]}
    if op == "quantize":
        sr.precond_quantize8(h, st["x"], q=st["q"], scale=st["s"], qt=st["qt"], scale_t=st["st"],
                             block=sr.BLOCK_TILE if case["block"] == "tile" else sr.BLOCK_ROW)
        return {k: st[k] for k in ("q", "s", "qt", "st") if st[k] is not None}
    if op == "gemm":
        sr.precond_gemm8(h, st["a"], st["as"], st["b"], st["bs"], st["out"], accumulate=case["accumulate"])
        return st["out"]
    sr.precond_distill(h, st["z"], st["ids"], st["t"], st["loss"], weight=st["weight"], temperature=case["tau"],
                       dlogits=st["dz"])
    return {"loss": st["loss"], "dlogits": st["dz"]} if case["grad"] else {"loss": st["loss"]}


def _run_plain(st):
    op, case = st["op"], st["case"]
    if op == "norm":
        h = st["x"]
        if case["residual"]:
            h = (h.float() + st["r"].float()).to(h.dtype)          # the stream keeps its type
        f = h.float()
        rstd = torch.rsqrt((f * f).mean(dim=1) + EPS)
        q, s = _to8(f * rstd[:, None] * st["w"], "row")
        out = {"q": q, "scale": s, "rstd": rstd}
        return dict(out, h=h) if case["residual"] else out
    if op == "norm_grad":
        dy, f, r = st["dy"].float(), st["x"].float(), st["rstd"][:, None]
        n = f * r
        g = dy * st["w"]
        dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
        if case["residual"]:
            dx = dx + st["dr"].float()
        return {"dx": dx.to(st["dy"].dtype), "dw": (dy * n).sum(dim=0)}
    if op == "quantize":
        f, out = st["x"].float(), {}
        if case["ways"] != "columns":
            out["q"], out["s"] = _to8(f, case["block"])
        if case["ways"] != "rows":
            out["qt"], out["st"] = _to8(f.t(), case["block"])
        return out
    if op == "gemm":
        c = _from8(st["a"], st["as"]) @ _from8(st["b"], st["bs"]).t()
        return st["out"].add_(c) if case["accumulate"] else c.to(TYPES[case["out"]])
    tau = case["tau"]
    z = st["z"].float() / tau
    live = st["ids"] >= 0
    ids = st["ids"].clamp(min=0)
    t = torch.where(live, st["t"] / tau, torch.full_like(st["t"], -math.inf))
    logp = t - torch.logsumexp(t, dim=1, keepdim=True)
    p = torch.where(live, torch.exp(logp), torch.zeros_like(t))
    m = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(dim=1, keepdim=True)
    logq = torch.gather(z, 1, ids) - m - torch.log(total)
    loss = tau * tau * st["weight"] * torch.where(live, p * (logp - logq), torch.zeros_like(p)).sum(dim=1)
    if not case["grad"]:
        return {"loss": loss}
    e.div_(total)
    e.scatter_add_(1, ids, -p)                                      # entries without a candidate add zero
    return {"loss": loss, "dlogits": e.mul_(tau * st["weight"][:, None]).to(st["z"].dtype)}


# --------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("norm", "norm_grad"):
        rows, cols, b = case["rows"], case["cols"], size[case["dtype"]]
        n = rows * cols
        if op == "norm":
            return {"bytes": n * (b * (3 if case["residual"] else 1) + 1) + rows * (cols / 128 + 4) + 4 * cols, "flops": 8 * n}
        return {"bytes": n * b * (4 if case["residual"] else 3) + 4 * rows + 8 * cols, "flops": 10 * n}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        ways = 2 if case["ways"] == "both" else 1
        return {"bytes": n * (size[case["dtype"]] + ways * (1 + 1 / 128)), "flops": 3 * n * ways}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        c = m * n * size[case["out"]] * (2 if case["accumulate"] else 1)
        return {"bytes": (m + n) * k * (1 + 1 / 128) + c, "flops": 2 * m * n * k}
    # rows of weight zero (one in eight) need no reading, and a zero gradient written
    n, b = case["rows"] * case["vocab"], size[case["dtype"]]
    return {"bytes": n * b * (0.875 + (1 if case["grad"] else 0)) + case["rows"] * (12 * case["top"] + 8), "flops": n * (6 if case["grad"] else 4)}


# --------------------------------------------------------------------------------------------- 64 bits
def _before8(x, block):
    """What an 8-bit matrix stands for, before its rounding: x over its block's scale, and the scales.  (A value in
    the middle of two 8-bit numbers goes either way with its last fp32 bit, so that the rounded ones say little.)"""
    rows, cols = x.shape
    blocks = -(-cols // 128)
    p = torch.nn.functional.pad(x, (0, blocks * 128 - cols)).view(rows, blocks, 128)
    amax = p.abs().amax(dim=2)
    if block == "tile":
        up = torch.nn.functional.pad(amax, (0, 0, 0, _pad_to(rows, 128) - rows)).view(-1, 128, blocks).amax(dim=1)
        amax = up.repeat_interleave(128, dim=0)[:rows]
    two_to = lambda k: ((k.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / E4M3_MAX))
    e = torch.where(amax > E4M3_MAX * two_to(e), e + 1, torch.where(amax <= E4M3_MAX * two_to(e - 1), e - 1, e))
    e = torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))
    s = torch.ones(_pad_to(rows, 128), _pad_to(blocks, 4), dtype=torch.float64, device=x.device)
    s[:rows, :blocks] = two_to(e)
    s = s.view(s.shape[0] // 128, 4, 32, s.shape[1] // 4, 4).permute(3, 0, 2, 1, 4)
    return (p / two_to(e)[:, :, None]).reshape(rows, blocks * 128)[:, :cols], s.contiguous()


def _values64(q, s):
    rows, cols = q.shape
    v = s.float().double().permute(1, 3, 2, 0, 4).reshape(s.shape[1] * 128, -1)[:rows]
    return q.float().double() * v[:, torch.arange(cols, device=q.device) // 128]


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
        rms = torch.sqrt(x.square().mean(dim=1) + EPS)
        # a block whose largest value is at the boundary of two scales goes with its last bit: no scale is given
        out["q"] = _before8(x / rms[:, None] * st["w"].double(), "row")[0]
        out["scale"], out["rstd"] = None, 1 / rms
        return out
    if op == "norm_grad":
        x, dy, w, r = st["x"].double(), st["dy"].double(), st["w"].double(), st["rstd"].double()
        dot = (dy * w * x).sum(dim=1)
        dx = dy * w * r[:, None] - x * (r ** 3 * dot / case["cols"])[:, None]
        if case["residual"]:
            dx = dx + st["dr"].double()
        return {"dx": dx, "dw": torch.einsum("tc,tc,t->c", dy, x, r)}
    if op == "quantize":
        x, out = st["x"].double(), {}
        if case["ways"] != "columns":
            out["q"], out["s"] = _before8(x, case["block"])
        if case["ways"] != "rows":
            out["qt"], out["st"] = _before8(x.t(), case["block"])
        return out
    if op == "gemm":
        c = torch.einsum("mk,nk->mn", _values64(st["a"], st["as"]), _values64(st["b"], st["bs"]))
        return c + st["out"].double() if case["accumulate"] else c
    tau, losses, grads = case["tau"], [], []
    for a in range(0, case["rows"], 512):                          # a few rows at a time: 64 bits of a large vocabulary
        z, ids, w = st["z"][a:a + 512].double() / tau, st["ids"][a:a + 512], st["weight"][a:a + 512].double()
        logq = z - torch.logsumexp(z, dim=1, keepdim=True)
        t = (st["t"][a:a + 512].double() / tau).masked_fill(ids < 0, -math.inf)
        logp = torch.log_softmax(t, dim=1)
        p = logp.exp()
        kl = torch.where(p > 0, p * (logp - logq.gather(1, ids.clamp(min=0))), torch.zeros_like(p)).sum(dim=1)
        losses.append(w * kl * tau ** 2)
        if case["grad"]:
            g = logq.exp_().scatter_add_(1, ids.clamp(min=0), -p)
            grads.append((g * (w * tau)[:, None]).to(torch.float32 if case["rows"] * case["vocab"] > 1e8 else torch.float64))
    out = {"loss": torch.cat(losses)}
    if case["grad"]:
        out["dlogits"] = torch.cat(grads)
    return out
