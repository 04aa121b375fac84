"""The clipped policy loss and its gradient on the GPU against the plain 64-bit form (training_plain.py).

Tolerances: E = 2^-24.  With x = (z - m) / tau the exponents of 2 are off by 4 E |x| (the constant, the division, the
fma and the shift's rounding), the powers by 2^-22, a row's sum by that and by vocab / 2048 + 64 additions one after
another; the far terms, whose |x| is large, are as much smaller.  So log q is off by 4 E (|x_id| + 8) + 2^-21 +
(vocab / 2048 + 64) E, called `t`; ratio and exp(d) by t of themselves, and the gradient's two factors by theirs."""
import math

import pytest
import torch

import operators_plain as P
import shampoo_roots_gb300 as sr
import training_plain as T

pytestmark = pytest.mark.gpu
E, E16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LOW, HIGH = 0.2, 0.28


@pytest.fixture(scope="module")
def pc():
    p = sr.Preconditioner(0)
    yield p
    p.close()


def inputs(rows, vocab, dtype, tau, seed=0, spread=2.5):
    """Logits, taken tokens, advantages, old and reference log probabilities and weights; no ratio lies near a bound."""
    g = P.generator(seed + rows * 31 + vocab)
    z = (spread * tau * P.randn(g, rows, vocab)).to(TYPES[dtype])
    ids = torch.randint(0, vocab, (rows,), generator=g)
    ids[::3] = z.float().argmax(dim=1)[::3]                         # likely ones too
    logp = torch.log_softmax(z.double() / tau, dim=1).gather(1, ids[:, None])[:, 0]
    step = 0.3 * P.randn(g, rows)
    for bound in (math.log(1 - LOW), math.log(1 + HIGH)):
        step = torch.where((step - bound).abs() < 1e-2, step + 3e-2, step)
    adv = P.randn(g, rows)
    weight = torch.rand(rows, generator=g) + 0.1
    return z, ids, adv, (logp - step).float(), (logp + 0.3 * P.randn(g, rows)).float(), weight


def check(pc, z, ids, adv, old, ref, weight, tau=1.0, kl=0.05, pitch=0, in_place=False, bits=64):
    rows, vocab = z.shape
    put = lambda t: None if t is None else t.cuda()
    place = (lambda t: P.pitched(t, vocab + pitch, offset=pitch % 5)) if pitch else (lambda t: t.cuda())
    dz_, ids_ = place(z), ids.to(torch.int32 if bits == 32 else torch.int64).cuda()
    loss, logp = torch.full((rows,), math.nan, device="cuda"), torch.full((rows,), math.nan, device="cuda")
    grad = dz_ if in_place else place(torch.full_like(z, math.nan))
    kw = dict(advantage=put(adv), old_logp=put(old), ref_logp=put(ref), weight=put(weight), temperature=tau, clip_low=LOW, clip_high=HIGH,
              kl=kl)
    before = None if in_place else dz_.clone()
    sr.precond_policy(pc.h, dz_, ids_, loss=loss, logp=logp, dlogits=grad, **kw)
    if before is not None:
        assert torch.equal(before, dz_)
    wl, ws, wg = T.policy(z, ids, adv, old, ref, weight, tau, LOW, HIGH, kl)
    live = ((ids >= 0) & (ids < vocab)) & (True if weight is None else weight != 0)
    x = z.double() / tau
    xid = torch.where(live, (x.gather(1, ids.clamp(0, vocab - 1)[:, None])[:, 0] - x.amax(dim=1)).abs(), torch.zeros(rows, dtype=torch.float64))
    t = 4 * E * (xid + 8) + 2.0 ** -21 + (vocab / 2048 + 64) * E
    assert bool(((logp.cpu().double() - ws).abs() <= t + E * ws.abs()).all())
    w = torch.ones(rows, dtype=torch.float64) if weight is None else weight.double()
    ratio = torch.ones(rows, dtype=torch.float64) if old is None else torch.exp(ws - old.double())
    ed = torch.exp(ref.double() - ws) if kl and ref is not None else torch.zeros(rows, dtype=torch.float64)
    by = t + 8 * E * (1 + ws.abs() + (0 if old is None else old.abs().double()) + (0 if ref is None else ref.abs().double()))
    size = w.abs() * (ratio * adv.double().abs() + kl * (ed + 1)) * live
    assert bool(((loss.cpu().double() - wl).abs() <= 2 * size * by + 1e-38).all())
    # |dz| = size / tau (q, or 1 - q at the taken token) at most, each factor off by `by`
    q = torch.softmax(x, dim=1)
    far = 4 * E * (x - x.amax(dim=1, keepdim=True)).abs() + 2.0 ** -20
    part = q.clone()
    part.scatter_(1, ids.clamp(0, vocab - 1)[:, None], 1 - q.gather(1, ids.clamp(0, vocab - 1)[:, None]))
    tol = (size / tau)[:, None] * part * (3 * by[:, None] + far) + 1e-38
    got = grad.cpu().double()
    bad = (got - wg).abs() > tol + (E16 * (wg.abs() + tol) if z.dtype == torch.bfloat16 else 0)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())
    assert bool((got[~live] == 0).all()) and bool((loss.cpu()[~live] == 0).all()) and bool((logp.cpu()[~live] == 0).all())
    if not in_place:                                                # the parts alone are the same
        l2, s2 = torch.empty_like(loss), torch.empty_like(loss)
        sr.precond_policy(pc.h, dz_, ids_, loss=l2, **kw)
        sr.precond_policy(pc.h, dz_, ids_, logp=s2, weight=put(weight), temperature=tau)
        assert torch.equal(l2, loss) and torch.equal(s2, logp)
    return loss, logp, grad


@pytest.mark.parametrize("rows,vocab", [(1, 1), (1, 2), (3, 7), (5, 64), (2, 500), (40, 513), (33, 1000), (17, 4099), (9, 32000), (5, 50001),
                                        (3, 131072), (2, 300001), (2, 140001), (1, 600001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy(pc, rows, vocab, dtype):
    check(pc, *inputs(rows, vocab, dtype, 1.0))
    z, ids, adv, old, ref, weight = inputs(rows, vocab, dtype, 0.7, seed=5)
    check(pc, z, ids, adv, None, None, None, tau=0.7, kl=0.0, bits=32)


@pytest.mark.parametrize("rows,vocab,dtype,pitch", [(400, 1000, "bf16", 0), (700, 333, "f32", 3), (350, 2047, "bf16", 1), (31, 50257, "bf16", 2),
                                                    (12, 70001, "f32", 1), (6, 400001, "bf16", 7), (5, 280003, "f32", 5), (320, 9000, "f32", 0), (5100, 130, "bf16", 0),
                                                    (5000, 70, "f32", 1), (40, 2048, "bf16", 0), (40, 2049, "bf16", 3), (60, 1024, "f32", 2),
                                                    (60, 50001, "bf16", 1), (90, 20003, "f32", 1), (25, 131072, "bf16", 0), (160, 5000, "bf16", 3),
                                                    (22, 140001, "f32", 1), (40, 300001, "bf16", 1), (320, 2050, "bf16", 0)])
def test_policy_layouts(pc, rows, vocab, dtype, pitch):
    """Rows at every alignment, on a warp that takes several, on 1 to 8 blocks, few and many of them, and read twice."""
    check(pc, *inputs(rows, vocab, dtype, 1.3), tau=1.3, pitch=pitch)


@pytest.mark.parametrize("rows,vocab,dtype", [(50, 1000, "bf16"), (9, 50001, "f32"), (3, 131072, "bf16"), (2, 300001, "f32"), (2, 700001, "bf16"), (2, 500003, "f32"),
                                              (200, 6001, "bf16"), (45, 50001, "bf16"), (3000, 100, "f32")])
def test_policy_in_place(pc, rows, vocab, dtype):
    a = inputs(rows, vocab, dtype, 1.0)
    one = check(pc, *a)
    two = check(pc, *a, in_place=True)
    for x, y in zip(one, two):
        assert torch.equal(x, y)


@pytest.mark.parametrize("rows,vocab,dtype,pitch", [(153, 2049, "bf16", 0), (153, 1025, "f32", 1), (160, 2500, "bf16", 3), (200, 6144, "bf16", 0),
                                                    (200, 6145, "bf16", 0), (608, 6001, "bf16", 5), (609, 6145, "bf16", 1), (609, 12288, "bf16", 0),
                                                    (609, 12289, "bf16", 0), (700, 4099, "f32", 2), (650, 6143, "f32", 1), (1201, 2001, "f32", 0),
                                                    (5003, 2055, "bf16", 1)])
def test_policy_middle_rows(pc, rows, vocab, dtype, pitch):
    """Rows of a warp in shared memory, at both ends of their lengths and numbers and at every alignment; in place as well."""
    a = inputs(rows, vocab, dtype, 0.9)
    one = check(pc, *a, tau=0.9, pitch=pitch)
    two = check(pc, *a, tau=0.9, pitch=pitch, in_place=True)
    for x, y in zip(one, two):
        assert torch.equal(x, y)
    z, ids, adv, old, ref, weight = a
    weight[::3], ids[1::7], ids[2::7] = 0, -1, vocab
    check(pc, z, ids, adv, old, ref, weight, tau=0.9, pitch=pitch)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_policy_middle_masks(pc, dtype):
    """Rows of a warp in shared memory: forbidden tokens, rows that are not read, what is not a number, a sure policy, the
    taken token at every place, and gradients beside the logits' vectors."""
    rows, vocab = 640, 2601
    z, _, adv, _, ref, weight = inputs(rows, vocab, "f32", 1.0, seed=3)
    z = z.to(TYPES[dtype])
    ids = (torch.arange(rows) * 61) % vocab
    ids[:40], ids[40:80] = torch.arange(40), vocab - 1 - torch.arange(40)
    z[:, 5::9] = -math.inf
    ids = torch.where(ids % 9 == 5, ids - 1, ids)
    z[100:110, :] = z[100:110, :].clamp(max=0.0)
    z[torch.arange(100, 110), ids[100:110]] = 90.0
    logp = torch.log_softmax(z.double(), dim=1).gather(1, ids[:, None])[:, 0].float()
    got = [torch.full(s, math.nan, device="cuda") for s in ((rows,), (rows,), (rows, vocab))]
    got[2] = got[2].to(TYPES[dtype])
    kw = dict(advantage=adv.cuda(), old_logp=(logp - 0.05).cuda(), clip_low=LOW, clip_high=HIGH)
    zz, at = z.clone(), ids.clone()
    zz[7], zz[8, 3], zz[9, 3], zz[10] = math.nan, math.nan, math.inf, math.nan
    weight[7], at[10] = 0.0, -1
    sr.precond_policy(pc.h, zz.cuda(), at.cuda(), loss=got[0], logp=got[1], dlogits=got[2], weight=weight.cuda(), **kw)
    wl, ws, wg = T.policy(z, ids, adv, logp - 0.05, None, weight, 1.0, LOW, HIGH, 0.0)
    loss, lp, grad = (t.cpu().double() for t in got)
    assert bool(lp[8:10].isnan().all()) and bool(grad[8:10].isnan().any(dim=1).all())
    for r in (7, 10):
        assert loss[r] == 0 and lp[r] == 0 and bool((grad[r] == 0).all())
    keep = torch.tensor([r for r in range(rows) if r not in (7, 8, 9, 10)])
    # log q by 4 E (|x| + 8) + 2^-21 + 66 E relative to 1, |x| < 128; the factors by that and E for each of their roundings
    by = 4 * E * 136 + 2.0 ** -21 + 66 * E
    assert bool(((lp - ws)[keep].abs() <= by + E * ws[keep].abs()).all())
    size = (weight.double() * math.exp(0.05) * adv.double().abs())[keep, None]
    tol = 8 * by * (size * (ids[keep, None] == torch.arange(vocab)) + wg[keep].abs()) + 1e-38
    assert bool(((grad - wg)[keep].abs() <= tol + (E16 * (wg[keep].abs() + tol) if dtype == "bf16" else 0)).all())
    assert bool((grad[keep][:, 5::9] == 0).all())
    one = got[2].clone()
    both = torch.zeros(rows, vocab + 3, dtype=z.dtype, device="cuda")
    sr.precond_policy(pc.h, zz.cuda(), at.cuda(), loss=got[0], dlogits=both[:, 3:], weight=weight.cuda(), **kw)
    assert torch.equal(both[:, 3:][keep.cuda()], one[keep.cuda()]) and bool((both[:, :3] == 0).all())


@pytest.mark.parametrize("vocab", [9, 700, 50001, 600001])
def test_policy_every_place(pc, vocab):
    """The taken token first, last, and beside every border of vectors, threads and blocks' parts."""
    at = sorted({0, 1, 7, 8, vocab // 2, vocab - 1, vocab - 2, vocab - 8, vocab - 9, min(vocab - 1, 4096), min(vocab - 1, 12512), min(vocab - 1, 75008),
                 min(vocab - 1, 75007)} & set(range(vocab)))
    z, _, adv, _, _, weight = inputs(len(at), vocab, "f32", 1.0, seed=2)
    ids = torch.tensor(at)
    logp = torch.log_softmax(z.double(), dim=1).gather(1, ids[:, None])[:, 0].float()
    check(pc, z, ids, adv, logp - 0.05, logp + 0.2, weight)
    check(pc, z, ids, adv, logp - 0.05, logp + 0.2, weight, pitch=1)


@pytest.mark.parametrize("vocab", [701, 3001, 40001])
def test_policy_masks(pc, vocab):
    """Rows of weight 0 and without a taken token are not read, whatever they hold; all rows masked; empty calls."""
    z, ids, adv, old, ref, weight = inputs(60, vocab, "f32", 1.0)
    weight[::4] = 0
    ids[1], ids[2], ids[3], ids[5] = -1, vocab, -100, 2 ** 40
    z[0], z[1], z[2] = math.nan, math.inf, -math.inf
    adv[0], old[0], ref[4] = math.nan, math.inf, math.nan
    live = ((ids >= 0) & (ids < vocab)) & (weight != 0)
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    loss, logp, grad = (torch.full(s, math.nan, device="cuda") for s in ((60,), (60,), (60, vocab)))
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=old.cuda(), ref_logp=ref.cuda(), weight=weight.cuda(), kl=0.1,
                      loss=loss, logp=logp, dlogits=grad)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad).all())
    assert bool((grad.cpu()[~live] == 0).all()) and bool((logp.cpu()[~live] == 0).all()) and bool((loss.cpu()[~live] == 0).all())
    assert bool((grad.cpu()[live] != 0).any(dim=1).any())
    keep = live.nonzero()[:, 0]
    check(pc, zz[keep], ids[keep], adv[keep], old[keep], ref[keep], weight[keep])
    check(pc, zz, ids.clamp(0, vocab - 1), adv.nan_to_num(), old.nan_to_num(posinf=0.0), ref.nan_to_num(), torch.zeros(60))
    e = torch.empty(0, vocab, device="cuda")
    none = torch.empty(0, device="cuda")
    sr.precond_policy(pc.h, e, torch.empty(0, dtype=torch.int64, device="cuda"), advantage=none, loss=none, dlogits=torch.empty_like(e))


@pytest.mark.parametrize("vocab", [1000, 5000])
def test_policy_masked_vocabulary(pc, vocab):
    """Forbidden tokens at -infinity or at the type's lowest value; a forbidden token that was taken all the same."""
    for dtype in ("bf16", "f32"):
        z, ids, adv, old, ref, weight = inputs(24, vocab, dtype, 1.0, seed=9)
        for low in (-math.inf, torch.finfo(TYPES[dtype]).min):
            m = z.clone()
            m[:, ::2] = low
            ids = ids // 2 * 2 + 1
            ids[ids >= vocab] = vocab - 1
            logp = torch.log_softmax(m.double(), dim=1).gather(1, ids[:, None])[:, 0].float()
            loss, lp, grad = (torch.full(s, math.nan, device="cuda") for s in ((24,), (24,), (24, vocab)))
            grad = grad.to(TYPES[dtype])
            sr.precond_policy(pc.h, m.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=(logp - 0.05).cuda(), loss=loss, logp=lp, dlogits=grad)
            assert bool(((lp.cpu() - logp).abs() <= 1e-4).all()) and bool(torch.isfinite(loss).all())
            assert bool((grad[:, ::2] == 0).all()) and bool(torch.isfinite(grad).all())
        m = z.clone()
        m[:, 7] = -math.inf
        ids[:] = 7
        sr.precond_policy(pc.h, m.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=old.cuda(), loss=loss, logp=lp, dlogits=grad)
        assert bool((lp == -math.inf).all())                        # the ratio is 0: nothing to pull on below the bound
        assert bool((grad == 0).all()) and bool(torch.isfinite(loss).all())


@pytest.mark.parametrize("vocab,times", [(1000, 1), (5000, 1), (5000, 30), (50001, 1), (50001, 8), (600001, 1)])
def test_policy_sure(pc, vocab, times):
    """A policy that is sure of the taken token: log q and 1 - q keep their digits, where 1 - q is far below fp32's step
    at 1 and where q is 1 to the last bit."""
    n = 6 * times
    z = torch.zeros(n, vocab)
    ids = torch.tensor([0, vocab - 1, vocab // 2, 3, 64, 8]).repeat(times)
    gap = torch.tensor([20.0, 30.0, 50.0, 80.0, 5.0, 200.0]).repeat(times)
    z[torch.arange(n), ids] = gap
    adv = torch.ones(n)
    loss, logp, grad = (torch.full(s, math.nan, device="cuda") for s in ((n,), (n,), (n, vocab)))
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), loss=loss, logp=logp, dlogits=grad)
    others = (vocab - 1) * torch.exp(-gap.double())
    want = -torch.log1p(others)
    # of the powers of 2; the rest is E a step, of which a thread's sum has vocab / 2048 + 64
    tol = 2.0 ** -20 + 4 * E * gap.double() + (vocab / 2048 + 64) * E
    assert bool(((logp.cpu().double() - want).abs() <= (tol + 16 * E) * want.abs() + 1e-38).all())
    one = grad.cpu().double()[torch.arange(n), ids]
    rest = -others / (1 + others)
    assert bool(((one - rest).abs() <= (tol + 16 * E) * rest.abs() + 1e-38).all())
    z[:, 1] = math.nan                                              # and what is not a number shows
    z[0, 1] = math.inf
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), loss=loss, logp=logp, dlogits=grad)
    assert bool(logp.isnan().all()) and bool(loss.isnan().all()) and bool(grad.isnan().any(dim=1).all())
    one = torch.full((3, vocab), -math.inf, device="cuda")
    sr.precond_policy(pc.h, one, torch.zeros(3, dtype=torch.int64, device="cuda"), logp=logp[:3])
    assert bool(logp[:3].isnan().all())


@pytest.mark.parametrize("vocab,dtype", [(700, "bf16"), (3001, "bf16"), (2003, "f32"), (50001, "f32"), (500003, "f32")])
def test_policy_gradient_elsewhere(pc, vocab, dtype):
    """Gradients whose rows begin at other places than the logits': beside vectors, odd pitches, a slice of the logits' own buffer."""
    z, ids, adv, old, ref, weight = inputs(9, vocab, dtype, 1.0, seed=4)
    one = check(pc, z, ids, adv, old, ref, weight)
    kw = dict(advantage=adv.cuda(), old_logp=old.cuda(), ref_logp=ref.cuda(), weight=weight.cuda(), clip_low=LOW, clip_high=HIGH, kl=0.05)
    for offset, pitch in ((1, 0), (3, 5), (0, 2)):
        dz = P.pitched(torch.zeros_like(z), vocab + pitch, offset=offset)
        loss = torch.empty(9, device="cuda")
        sr.precond_policy(pc.h, z.cuda(), ids.cuda(), loss=loss, dlogits=dz, **kw)
        assert torch.equal(loss, one[0]) and torch.equal(dz, one[2])
    both = torch.zeros(9, 2 * vocab + 1, dtype=z.dtype, device="cuda")
    both[:, :vocab] = z.cuda()
    sr.precond_policy(pc.h, both[:, :vocab], ids.cuda(), loss=loss, dlogits=both[:, vocab + 1:], **kw)
    assert bool((both[:, vocab] == 0).all()) and torch.equal(both[:, :vocab], z.cuda())
    # the rows' vectors begin elsewhere, so that sums are joined in another order
    tol = 1e-5 * one[2].abs().float() + 2.0 ** -7 * (one[2].abs().float() if dtype == "bf16" else 0) + 1e-9
    assert bool(((both[:, vocab + 1:].float() - one[2].float()).abs() <= tol).all())


def test_policy_bounds(pc):
    """Which side of a bound passes a gradient, for each sign of the advantage; wide open and shut bounds."""
    vocab = 300
    z = P.randn(P.generator(4), 8, vocab)
    ids = torch.arange(8)
    logp = torch.log_softmax(z.double(), dim=1).gather(1, ids[:, None])[:, 0]
    step = torch.tensor([0.5, 0.5, -0.5, -0.5, 0.1, 0.1, -0.1, -0.1]).double()
    adv = torch.tensor([1.0, -1.0] * 4)
    for low, high in ((0.2, 0.2), (1.0, math.inf), (0.0, 0.0)):
        loss, grad = torch.empty(8, device="cuda"), torch.empty(8, vocab, device="cuda")
        sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=(logp - step).float().cuda(), clip_low=low, clip_high=high,
                          loss=loss, dlogits=grad)
        r = torch.exp(step)
        stopped = ((adv > 0) & (r > 1 + high)) | ((adv < 0) & (r < 1 - low))
        assert torch.equal((grad.cpu() == 0).all(dim=1), stopped)
        want = -torch.minimum(r * adv, r.clamp(1 - low, 1 + high) * adv)
        assert bool(((loss.cpu().double() - want).abs() <= 1e-5).all())


def test_policy_against_differences(pc):
    """<dz, u> against central differences of the 64-bit loss along random directions."""
    z, ids, adv, old, ref, weight = inputs(12, 400, "f32", 1.0, seed=3)
    loss, grad = torch.empty(12, device="cuda"), torch.empty(12, 400, device="cuda")
    sr.precond_policy(pc.h, z.cuda(), ids.cuda(), advantage=adv.cuda(), old_logp=old.cuda(), ref_logp=ref.cuda(), weight=weight.cuda(),
                      clip_low=LOW, clip_high=HIGH, kl=0.3, loss=loss, dlogits=grad)
    f = lambda x: float(T.policy(x, ids, adv, old, ref, weight, 1.0, LOW, HIGH, 0.3)[0].sum())
    g, step = P.generator(8), 1e-5
    for _ in range(4):
        u = P.randn(g, 12, 400).double()
        along = (f(z.double() + step * u) - f(z.double() - step * u)) / (2 * step)
        assert abs(float((grad.cpu().double() * u).sum()) - along) <= 1e-4


def test_policy_large_logits(pc):
    """Logits around 1e5 and -1e5: shifts whose product with log2(e) / tau is rounded."""
    for centre in (1e5, -1e5, 3e6):
        z, ids, adv, old, ref, weight = inputs(20, 4000, "f32", 1.0, seed=7)
        z = z + centre
        x = z.double()
        logp = torch.log_softmax(x, dim=1).gather(1, ids[:, None])[:, 0]
        check(pc, z, ids, adv, logp.float() - 0.05, logp.float() + 0.1, weight)


def test_preference_of_pairs(pc):
    """A preference loss over pairs of sequences by two calls: log probabilities, then their coefficients."""
    rows, vocab, beta = 40, 900, 0.1
    z, ids, _, _, ref, _ = inputs(rows, vocab, "f32", 1.0, seed=11)
    sequence = torch.arange(rows) // 10                              # 2 pairs: 0 over 1, 2 over 3
    dz, dids = z.cuda(), ids.cuda()
    logp, grad = torch.empty(rows, device="cuda"), torch.empty(rows, vocab, device="cuda")
    sr.precond_policy(pc.h, dz, dids, logp=logp)
    ratio = torch.zeros(4, device="cuda").index_add_(0, sequence.cuda(), logp - ref.cuda())
    push = beta * torch.sigmoid(-beta * (ratio[0::2] - ratio[1::2]))
    sr.precond_policy(pc.h, dz, dids, advantage=torch.stack((push, -push), 1).view(-1)[sequence.cuda()], dlogits=grad)
    x = z.double().requires_grad_()
    s = torch.log_softmax(x, dim=1).gather(1, ids[:, None])[:, 0] - ref.double()
    r = torch.zeros(4, dtype=torch.float64).index_add(0, sequence, s)
    (-torch.nn.functional.logsigmoid(beta * (r[0::2] - r[1::2]))).sum().backward()
    # the margin is a sum of 20 log probabilities, each within 2e-6; beta times that moves the sigmoid
    assert bool(((grad.cpu().double() - x.grad).abs() <= 1e-5 * x.grad.abs() + 1e-9).all())


def test_policy_captured_and_two_streams(pc):
    a = [t.cuda() for t in inputs(300, 20000, "bf16", 1.0)]
    z, ids, adv, old, ref, weight = a
    out = [[torch.empty(300, device="cuda"), torch.empty(300, device="cuda"), torch.empty_like(z)] for _ in range(3)]

    def call(o):
        sr.precond_policy(pc.h, z, ids, advantage=adv, old_logp=old, ref_logp=ref, weight=weight, kl=0.1, loss=o[0], logp=o[1], dlogits=o[2])

    call(out[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, o in zip(streams, out[1:]):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                call(o)
    torch.cuda.synchronize()
    for o in out[1:]:
        for x, y in zip(out[0], o):
            assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out[1])
    z.mul_(0.5)
    graph.replay()
    call(out[2])
    torch.cuda.synchronize()
    for x, y in zip(out[1], out[2]):
        assert torch.equal(x, y)
