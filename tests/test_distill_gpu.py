"""The distillation loss and its gradient against binary64.

Tolerances.  A row's sums take exponentials of t = (z - max) k whose rounding is
2^-24 |t|: weighted by 2^t that is at most 2^-23 of the sum, and a thread's and
a wave's partial sums of at most some 70 terms each add 70 2^-24 at the very
most: 2^-17 of each sum, and as much absolute in its logarithm.  k itself is
rounded by 2^-24, which moves a loss by 2^-24 times the largest cross term
sum p |d|.  The loss is rounded once.  A gradient's q takes 2^-17 of itself
from its sum and (|t| + 8) 2^-22 from its own exponential; p (|log p| + 8)
2^-23; the result half a step of its type, 2^-24 or 2^-8."""
import math

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = {torch.float32: 2.0 ** -24, BF: 2.0 ** -8}


def reference(z, ids, t, temperature, rest, g):
    """loss, its tolerance, gradient, its tolerance; by the formulas, in binary64 on the CPU, row by row."""
    z, ids, t, g = z.detach().double().cpu(), ids.cpu().long(), t.double().cpu(), g.double().cpu()
    n, v = z.shape
    c = 1.0 / temperature
    loss, dz = torch.zeros(n, dtype=torch.float64), torch.zeros(n, v, dtype=torch.float64)
    tl, tg = torch.zeros(n, dtype=torch.float64), torch.zeros(n, v, dtype=torch.float64)
    for r in range(n):
        ok = (ids[r] >= 0) & (ids[r] < v)
        at, tt = ids[r][ok], t[r][ok]
        p = torch.exp(tt)
        mass = p.sum()
        if not len(at) or mass == 0:
            continue
        if (z[r] == -math.inf).all():
            loss[r] = math.inf
            continue
        lq = torch.log_softmax(z[r] * c, 0)
        q = lq.exp()
        if rest == "renormalize":
            p, tt = p / mass, tt - mass.log()
        pv = torch.zeros(v, dtype=torch.float64).index_add(0, at, p)
        hit = torch.zeros(v, dtype=torch.bool)
        hit[at] = True
        on = p > 0
        loss[r] = (p[on] * (tt[on] - lq[at[on]])).sum()
        span = ((z[r] - z[r].max()) * c).clamp_min(-1e30).abs()
        own = span / math.log(2)
        cross = (p[on] * span[at[on]]).sum()
        coef = torch.ones(v, dtype=torch.float64)
        part = torch.ones(v, dtype=torch.float64)
        if rest == "bucket":
            left = (1.0 - mass).clamp_min(0.0)
            lr = torch.logsumexp(lq.masked_fill(hit, -math.inf), 0)
            if left > 0 and lr > -math.inf:
                loss[r] += left * (left.log() - lr)
                cross = cross + left * lr.abs()
                # shares of the others, from their own logits: against the row's, a far lr keeps nothing of log(count)
                other = torch.softmax((z[r] * c).masked_fill(hit, -math.inf), 0)
                dz[r] = g[r] * c * torch.where(hit, q - pv, other * (lr.exp() - left))
                part = torch.where(hit, q, other * (lr.exp() + left))
                own = torch.where(hit, own, (lq - lq.masked_fill(hit, -math.inf).max()).clamp_min(-1e30).abs() / math.log(2))
            else:
                dz[r] = g[r] * c * (mass * q - pv)
                part = q
        else:
            dz[r] = g[r] * c * (q - pv)
            part = q
        tl[r] = 2.0 ** -17 + 2.0 ** -22 * (cross + loss[r].abs())
        pl = torch.zeros(v, dtype=torch.float64).index_add(0, at, p * (tt.clamp_min(-1e4).abs() + 8.0))
        tg[r] = g[r].abs() * c * (part * (2.0 ** -16 + (own.clamp_max(1e6) + 8.0) * 2.0 ** -21) + pl * 2.0 ** -22)
        del coef
    return loss, tl, dz, tg


def check(z, ids, t, temperature=1.0, rest="bucket", g=None, out=None):
    n = z.shape[0]
    if g is None:
        g = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) + 0.5
    loss, tl, dz, tg = reference(z, ids, t, temperature, rest, g)
    f = fq.fp4_distill_loss(z, ids, t, temperature=temperature, rest=rest)
    got = f.loss.double().cpu()
    same = (got == loss) | ((got - loss).abs() <= tl)
    assert same.all(), (got[~same][:4], loss[~same][:4], tl[~same][:4])
    d = fq.fp4_distill_loss_backward(z, ids, t, f, g, temperature=temperature, rest=rest, out=out)
    gd = d.double().cpu()
    bad = ~((gd - dz).abs() <= tg + HALF[z.dtype] * dz.abs() + 1e-37)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0], gd[bad][:3], dz[bad][:3], tg[bad][:3])
    return f, d


def teacher(z, top, temperature, noise, seed):
    """A teacher's own top list, as fp4_token_logprobs gives it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tz = z.float() + noise * torch.randn(z.shape, generator=g, device="cuda")
    if top <= 32:
        f = fq.fp4_token_logprobs(tz, temperature=temperature, top=top)
        return f.top_ids, f.top_logprobs
    lp = torch.log_softmax(tz / temperature, -1)
    v, i = torch.topk(lp, top)
    return i.to(torch.int32), v.contiguous()


def student(n, v, seed, dtype, sharp=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = 2.0 * torch.randn(n, v, generator=g, device="cuda")
    z[torch.arange(n, device="cuda"), torch.randint(0, v, (n,), generator=g, device="cuda")] += sharp
    return z.to(dtype)


@pytest.mark.parametrize("rest", ["bucket", "renormalize"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("n,v,top", [(1, 2, 1), (3, 7, 2), (1, 300, 32), (2, 1027, 5), (61, 5003, 8), (1, 50257, 20), (5, 40000, 128),
                                     (520, 700, 64), (3, 300007, 17), (2, 600011, 9)])
def test_loss_and_gradient(n, v, top, dtype, rest):
    z = student(n, v, n + v, dtype)
    for temperature in (1.0, 2.0, 0.7):
        ids, t = teacher(z, top, temperature, 0.5, v)
        check(z, ids, t, temperature, rest)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("start", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("v", [1, 5, 9, 33, 260, 4099, 20001])
def test_rows_at_any_element(dtype, start, v):
    """Rows that start and end anywhere, the listed tokens at both ends among them."""
    n = 4
    wide = student(n, v + 13, 5 + v, dtype)
    z = wide[:, start:start + v]
    top = min(6, v)
    ids = torch.stack([torch.randperm(v, device="cuda")[:top] for _ in range(n)]).to(torch.int32)
    ids[0, 0], ids[0, -1] = 0, v - 1
    ids[1, 0] = v // 2
    t = torch.log_softmax(torch.randn(n, top + 1, device="cuda"), -1)[:, :top].contiguous()
    check(z, ids, t)
    # a gradient into rows of another alignment, and in place
    out = torch.zeros(n, v + 9, dtype=dtype, device="cuda")
    _, d = check(z, ids, t, out=out[:, 2:2 + v])
    assert (out[:, :2] == 0).all() and (out[:, 2 + v:] == 0).all()
    own = wide.clone()
    view = own[:, start:start + v]
    f = fq.fp4_distill_loss(view, ids, t)
    g = torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) + 0.5
    fq.fp4_distill_loss_backward(view, ids, t, f, g, out=view)
    assert torch.equal(view, d)
    assert torch.equal(own[:, :start], wide[:, :start]) and torch.equal(own[:, start + v:], wide[:, start + v:])


@pytest.mark.parametrize("rest", ["bucket", "renormalize"])
def test_lists_with_gaps_and_repeats(rest):
    z = student(6, 500, 3, torch.float32)
    ids, t = teacher(z, 5, 1.0, 0.3, 4)
    ids, t = ids.clone(), t.clone()
    ids[0] = -1                                              # a padded row
    ids[1, 2] = -100                                         # a gap
    ids[1, 4] = 500                                          # just outside
    ids[2, 3] = ids[2, 0]                                    # listed twice
    ids[3] = ids[3, 0]                                       # five times the same
    t[3] -= 2.0
    t[4] = -math.inf                                         # no probability at all
    t[5, 1] = -math.inf
    f, d = check(z, ids, t, rest=rest)
    assert f.loss[0] == 0 and f.loss[4] == 0 and (d[0] == 0).all() and (d[4] == 0).all()


def test_the_whole_vocabulary_listed():
    """Nothing is left outside: the bucket's second term is gone, and a list that adds to 1 leaves q - p."""
    z = student(4, 9, 6, torch.float32)
    t = torch.log_softmax(torch.randn(4, 9, device="cuda"), -1)
    ids = torch.arange(9, device="cuda", dtype=torch.int32).repeat(4, 1)
    check(z, ids, t)
    check(z, ids, (t - 0.1).contiguous())                    # and one that does not
    check(z, ids, (t - 0.1).contiguous(), rest="renormalize")


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_confident_and_far_rows(dtype):
    """The others' probability far below binary32's range, both ways; huge logits; temperatures near zero."""
    z = torch.randn(5, 3000, device="cuda")
    ids = torch.tensor([[7, 11, 13]], dtype=torch.int32, device="cuda").repeat(5, 1)
    t = torch.log(torch.tensor([0.5, 0.3, 0.1], device="cuda")).repeat(5, 1).contiguous()
    z[0, [7, 11, 13]] += 400.0                               # R about e^-390
    z[1, 100] += 300.0                                       # the listed tokens about e^-300
    z[2] += 1e4
    z[3] *= 1e3
    z[4, 7] = 90.0
    check(z.to(dtype), ids, t)
    check(z.to(dtype), ids, t, rest="renormalize")
    check(z.to(dtype), ids, t, temperature=1e-3)
    check((z * 1e20).to(dtype), ids, t, temperature=3.0)


def test_masked_student():
    z = student(4, 600, 8, torch.float32)
    ids, t = teacher(z, 4, 1.0, 0.3, 9)
    inside = torch.zeros(4, 600, dtype=torch.bool, device="cuda").scatter(1, ids.long(), True)
    z[0] = torch.where(inside[0], z[0], -math.inf)           # nothing outside the list
    z[1, ids[1, 2].long()] = -math.inf                       # a listed token that the student cannot give
    z[2] = -math.inf                                         # nothing at all
    z[3, 100:500] = torch.where(inside[3, 100:500], z[3, 100:500], -math.inf)
    for rest in ("bucket", "renormalize"):
        f, d = check(z, ids, t, rest=rest)
        assert f.loss[1] == math.inf and f.loss[2] == math.inf and (d[2] == 0).all() and torch.isfinite(d).all()
    low = torch.finfo(torch.float32).min
    check(torch.where(torch.isinf(z), low, z)[[0, 1, 3]], ids[[0, 1, 3]], t[[0, 1, 3]])


def test_nan_and_infinity_stay_in_their_rows():
    z = student(5, 700, 10, torch.float32)
    ids, t = teacher(z, 4, 1.0, 0.3, 11)
    clean = fq.fp4_distill_loss(z, ids, t).loss
    bad = z.clone()
    bad[1, 650], bad[2, ids[2, 1].long()], bad[3, 3] = float("nan"), float("nan"), float("inf")
    f = fq.fp4_distill_loss(bad, ids, t)
    assert torch.isnan(f.loss[1:4]).all() and torch.equal(f.loss[[0, 4]], clean[[0, 4]])
    g = torch.ones(5, device="cuda")
    d = fq.fp4_distill_loss_backward(bad, ids, t, f, g)
    assert torch.isfinite(d[[0, 4]]).all() and torch.isnan(d[1:4]).any(1).all()
    # a row without a gradient is zeros whatever its logits hold
    g[1:4] = 0.0
    assert (fq.fp4_distill_loss_backward(bad, ids, t, f, g)[1:4] == 0).all()


@pytest.mark.parametrize("rest", ["bucket", "renormalize"])
@pytest.mark.parametrize("v", [700, 140001])                 # a row in one piece, and in several
def test_a_listed_nan_in_a_row_of_masks(v, rest):
    """A NaN logit that is listed makes the loss NaN also where every other logit is -inf; a row without entries keeps 0."""
    z = torch.full((4, v), -math.inf, device="cuda")
    z[0, 5], z[1, 9], z[3, 5] = float("nan"), float("nan"), float("nan")
    ids = torch.tensor([[5, 7], [5, 7], [5, 7], [-1, -1]], dtype=torch.int32, device="cuda")
    t = torch.log(torch.tensor([0.5, 0.25], device="cuda")).repeat(4, 1).contiguous()
    f = fq.fp4_distill_loss(z, ids, t, rest=rest)
    assert torch.isnan(f.loss[:2]).all() and f.loss[2] == math.inf and f.loss[3] == 0
    d = fq.fp4_distill_loss_backward(z, ids, t, f, torch.ones(4, device="cuda"), rest=rest)
    assert torch.isnan(d[:2]).any(1).all() and (d[2:] == 0).all()


@pytest.mark.parametrize("rest", ["bucket", "renormalize"])
@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_gradient_against_differences(rest, temperature):
    """Along a direction u with |u| <= 1 and h = 2^-6: central differences of
    the loss are h^2 / 6 times a third derivative off, which the third
    cumulants of u under q (below 1 for |u| <= 1, listed and outside) keep
    under 4 c^3, so 4 h^2 / 6 < 2^-12; two losses off by 2^-17 each give
    2^-17 / h = 2^-11."""
    z = student(8, 2000, 12, torch.float32, sharp=3.0)
    ids, t = teacher(z, 8, temperature, 0.5, 13)
    g = torch.ones(8, device="cuda")
    d = fq.fp4_distill_loss_backward(z, ids, t, fq.fp4_distill_loss(z, ids, t, temperature, rest), g, temperature, rest)
    for seed in range(3):
        u = torch.rand(8, 2000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * 2 - 1
        h = 2.0 ** -6
        up, dn = (fq.fp4_distill_loss(z + s * h * u, ids, t, temperature, rest).loss.double() for s in (1, -1))
        assert ((up - dn) / (2 * h) - (d.double() * u.double()).sum(1)).abs().max() < 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -14


def test_a_students_own_list_costs_nothing():
    """A teacher that is the student: the loss is zero within its tolerance, and so is the gradient's sum."""
    z = student(30, 4000, 14, torch.float32)
    ids, t = teacher(z, 32, 1.0, 0.0, 15)
    f, d = check(z, ids, t)
    assert (f.loss.abs() < 2.0 ** -15).all() and (d.double().sum(1).abs() < 2.0 ** -12).all()


def test_bits_repeat_and_rows_of_none():
    z = student(40, 30000, 16, BF)
    ids, t = teacher(z, 16, 1.0, 0.5, 17)
    f = fq.fp4_distill_loss(z, ids, t)
    for _ in range(3):
        assert torch.equal(fq.fp4_distill_loss(z, ids, t).loss, f.loss)
    e = fq.fp4_distill_loss(z[:0], ids[:0], t[:0])
    assert e.loss.shape == (0,)
    assert fq.fp4_distill_loss_backward(z[:0], ids[:0], t[:0], e, e.loss).shape == (0, 30000)
