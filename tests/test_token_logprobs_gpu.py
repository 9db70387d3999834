"""Token log probabilities, entropy and top alternatives, and the gradient of
the logits, against binary64.

Tolerances: exp((z - m) c) is taken as a power of two of a product with three
binary32 roundings, so its relative error is at most about 3 * 2^-24 |d| +
2^-23, and the terms that matter have |d| < 30: 6e-6.  A thread adds at most
vocab / 256 terms (below 600 here: 600 * 2^-24 = 3.6e-5 at the very worst,
all roundings one way), so log s and the entropy are within 5e-5 absolute,
plus 2^-22 of the magnitude for the final subtractions.  The gradient's p has
that relative error too."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
F = torch.float64
INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _reference(z, tokens, temp, top):
    top_z = z.to(F).amax(-1, keepdim=True)
    # the maximum is subtracted first: beside a logit of 1e38, binary64 would lose log s
    d = (z.to(F) - top_z.masked_fill(top_z == -INF, 0)) / temp
    lp = d - torch.logsumexp(d, -1, keepdim=True)
    p = lp.exp()
    ent = -(p * lp.masked_fill(p == 0, 0)).sum(-1)
    empty = (z == -INF).all(-1)
    lp[empty], p[empty], ent[empty] = -INF, 0.0, 0.0
    ok = (tokens >= 0) & (tokens < z.shape[1])
    hit = lp.gather(1, tokens.clamp(0, z.shape[1] - 1)[:, None])[:, 0]
    hit = torch.where(ok, hit, torch.zeros_like(hit))
    ids = torch.sort(z.float() + 0.0, dim=-1, descending=True, stable=True).indices[:, :top]
    return hit, ent, ids, lp.gather(1, ids), lp, p, ok


def _near(got, want, what):
    got, want = got.cpu().to(F), want.float().to(F)       # -6.8e38 (the lowest logit at temperature 1/2) is -inf in binary32
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = torch.where(same, torch.zeros_like(want), (got - want).abs())
    tol = 5e-5 + want.abs().nan_to_num(0, 0, 0) * 2.0 ** -22
    assert not (~(off <= tol)).any(), (what, float(off.nan_to_num(1e9).max()))


def _check(z, tokens, temp=1.0, top=0, grads=True, seed=0):
    zd = z.cuda() if z.device.type == "cpu" else z
    z = zd.cpu()
    f = fq.fp4_token_logprobs(zd, tokens.cuda(), temperature=temp, top=top)
    hit, ent, ids, best, lp, p, ok = _reference(z, tokens, temp, top)
    _near(f.logprob, hit, "logprob")
    _near(f.entropy, ent, "entropy")
    if top:
        assert torch.equal(f.top_ids.cpu().long(), ids)
        _near(f.top_logprobs, best, "top_logprobs")
    if not grads:
        return f
    g = torch.Generator().manual_seed(seed)
    gl, ge = torch.randn(len(z), generator=g), torch.randn(len(z), generator=g)
    for a, b in ((gl, ge), (gl, None), (None, ge)):
        dz = fq.fp4_token_logprobs_backward(zd, tokens.cuda(), f, None if a is None else a.cuda(),
                                            None if b is None else b.cuda(), temperature=temp).cpu()
        gl64 = torch.where(ok, a.to(F), 0.0) if a is not None else torch.zeros(len(z), dtype=F)
        ge64 = b.to(F) if b is not None else torch.zeros(len(z), dtype=F)
        empty = (z == -INF).all(-1)
        gl64, ge64 = gl64.masked_fill(empty, 0)[:, None], ge64.masked_fill(empty, 0)[:, None]
        one = torch.nn.functional.one_hot(tokens.clamp(0, z.shape[1] - 1), z.shape[1]) * ok[:, None]
        l0 = lp.masked_fill(p == 0, 0)
        want = (gl64 * (one - p) - ge64 * p * (l0 + ent[:, None])) / temp
        mag = (gl64.abs() * p + ge64.abs() * p * (l0.abs() + ent[:, None] + 1)) / temp
        half = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -23
        off = (dz.to(F) - want).abs()
        tol = 1e-4 * mag + half * (want.abs() + gl64.abs() * one / temp) + 1e-37
        assert not (~(off <= tol)).any(), (float(off.max()), (~(off <= tol)).nonzero()[0].tolist())
    return f


def _tokens(g, n, v):
    t = torch.randint(0, v, (n,), generator=g)
    if n > 3:
        t[1], t[2], t[3] = -100, v, -1
    return t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v,top", [(1, 1, 1), (1, 2, 2), (5, 7, 3), (4, 33, 32), (2, 100, 0), (6, 257, 20), (3, 1000, 5),
                                     (1, 8191, 32), (2, 8200, 20), (70, 8192, 1), (1, 50257, 20), (600, 515, 4),
                                     (520, 2050, 0), (3, 140001, 20)])
def test_random_rows(dtype, n, v, top):
    g = torch.Generator().manual_seed(n * 1000 + v)
    z = (torch.randn(n, v, generator=g) * 3).to(dtype)
    _check(z, _tokens(g, n, v), [1.0, 0.6, 1.7][v % 3], min(top, v))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pieces", [False, True])
def test_orders_ties_and_masks(dtype, pieces):
    """Rows in falling and rising order (every element a new maximum), of one
    value, with few distinct values (ties go to the lowest index), with most
    entries masked, fewer finite entries than alternatives asked for, the
    type's lowest value as a mask, zeros of both signs."""
    v = 20000 if pieces else 3000
    n = 9 if pieces else 513
    g = torch.Generator().manual_seed(v)
    z = (torch.randn(n, v, generator=g) * 2)
    z[0] = torch.linspace(9, -9, v)
    z[1] = torch.linspace(-9, 9, v)
    z[2] = 1.25
    z[3] = torch.randint(0, 3, (v,), generator=g).float()
    z[4][torch.rand(v, generator=g) < 0.99] = -INF
    z[5] = -INF
    z[5][[7, v - 1]] = torch.tensor([0.5, 0.25])
    low = torch.finfo(dtype).min
    z = z.to(dtype)
    z[6][torch.rand(v, generator=g) < 0.9] = low
    z[7] = low
    z[8] = 0.0
    z[8][::3] = -0.0
    tok = torch.randint(0, v, (n,), generator=g)
    tok[5] = 7
    for temp in (1.0, 0.5):
        _check(z, tok, temp, 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v", [(6, 9000), (515, 700)])
def test_empty_rows_and_values_that_are_no_numbers(dtype, n, v):
    g = torch.Generator().manual_seed(v)
    z = (torch.randn(n, v, generator=g)).to(dtype)
    z[0] = -INF
    z[1][v // 2] = float("nan")
    z[2][5] = INF
    z[3] = float("nan")
    tok = torch.randint(0, v, (n,), generator=g)
    zd = z.cuda()
    f = fq.fp4_token_logprobs(zd, tok.cuda(), top=4)
    assert f.logprob[0] == -INF and f.entropy[0] == 0
    assert f.top_ids[0].tolist() == [0, 1, 2, 3] and (f.top_logprobs[0] == -INF).all()
    for r in (1, 2, 3):
        assert torch.isnan(f.logprob[r]) and torch.isnan(f.entropy[r])
    assert int(f.top_ids[1][0]) == v // 2 and int(f.top_ids[2][0]) == 5 and f.top_ids[3].tolist() == [0, 1, 2, 3]
    one = torch.ones(n, device="cuda")
    dz = fq.fp4_token_logprobs_backward(zd, tok.cuda(), f, one, one)
    assert (dz[0] == 0).all()
    assert torch.isnan(dz[1][0]) and torch.isfinite(dz[4:].float()).all()
    _check(z[4:], tok[4:], top=4)
    # padding: no token and no entropy gradient gives zeros whatever the row holds
    pad = tok.clone()
    pad[:4] = -100
    f = fq.fp4_token_logprobs(zd, pad.cuda())
    dz = fq.fp4_token_logprobs_backward(zd, pad.cuda(), f, one)
    assert (dz[:4] == 0).all() and (f.logprob[:4] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [1, 3, 8])
def test_rows_at_any_element(dtype, shift):
    g = torch.Generator().manual_seed(shift)
    wide = (torch.randn(5, 9011, generator=g) * 2).to(dtype).cuda()
    z = wide[:, shift:shift + 8999]
    tok = torch.randint(0, 8999, (5,), generator=g)
    _check(z, tok, 0.8, 7)
    f = fq.fp4_token_logprobs(z, tok.cuda(), temperature=0.8)
    gl = torch.randn(5, generator=g).cuda()
    want = fq.fp4_token_logprobs_backward(z, tok.cuda(), f, gl, temperature=0.8)
    out = torch.full((5, 9020), 7.0, dtype=dtype, device="cuda")
    fq.fp4_token_logprobs_backward(z, tok.cuda(), f, gl, temperature=0.8, out=out[:, 2:2 + 8999])
    assert torch.equal(out[:, 2:2 + 8999], want) and (out[:, :2] == 7).all() and (out[:, 9001:] == 7).all()
    keep = wide.clone()
    fq.fp4_token_logprobs_backward(z, tok.cuda(), f, gl, temperature=0.8, out=z)       # in place
    assert torch.equal(z, want) and torch.equal(wide[:, :shift], keep[:, :shift])
    assert torch.equal(wide[:, shift + 8999:], keep[:, shift + 8999:])


def test_gradient_against_differences():
    """The loss sum(gl logprob + ge entropy) in binary64, central differences
    of step 1e-4 along random directions: the truncation error is of order
    1e-8 of third derivatives of order one."""
    g = torch.Generator().manual_seed(2)
    n, v, temp = 6, 300, 0.9
    z = (torch.randn(n, v, generator=g) * 2)
    tok = torch.randint(0, v, (n,), generator=g)
    gl, ge = torch.randn(n, generator=g), torch.randn(n, generator=g)
    zd = z.cuda()
    f = fq.fp4_token_logprobs(zd, tok.cuda(), temperature=temp)
    dz = fq.fp4_token_logprobs_backward(zd, tok.cuda(), f, gl.cuda(), ge.cuda(), temperature=temp).cpu().to(F)

    def loss(zz):
        lp = torch.log_softmax(zz / temp, -1)
        return float((gl.to(F) * lp[torch.arange(n), tok] - ge.to(F) * (lp.exp() * lp).sum(-1)).sum())

    for _ in range(4):
        d = torch.randn(n, v, generator=g, dtype=F)
        want = (loss(z.to(F) + 1e-4 * d) - loss(z.to(F) - 1e-4 * d)) / 2e-4
        assert abs(float((dz * d).sum()) - want) <= 1e-4 * float((dz.abs() * d.abs()).sum()) + 1e-6


def test_no_tokens_empty_batch_and_replay():
    g = torch.Generator().manual_seed(4)
    z = torch.randn(3, 9000, generator=g).cuda()
    f = fq.fp4_token_logprobs(z, top=3)
    assert f.logprob is None
    _near(f.entropy, _reference(z.cpu(), torch.zeros(3, dtype=torch.long), 1.0, 3)[1], "entropy")
    e = fq.fp4_token_logprobs(z[:0], torch.empty(0, dtype=torch.long, device="cuda"), top=2)
    assert e.logprob.shape == (0,) and e.top_ids.shape == (0, 2)
    assert fq.fp4_token_logprobs_backward(z[:0], None, fq.fp4_token_logprobs(z[:0])).shape == (0, 9000)
    tok = torch.randint(0, 9000, (3,), generator=g).cuda()
    gl = torch.randn(3, generator=g).cuda()

    def step(stream=None):
        f = fq.fp4_token_logprobs(z, tok, top=5, stream=stream)
        return (f.logprob, f.entropy, f.top_ids, f.top_logprobs,
                fq.fp4_token_logprobs_backward(z, tok, f, gl, gl, stream=stream))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """More than 2^31 logits: rows of zeros, whose results are known, and three
    last rows like any others; then rows far apart in one allocation."""
    g = torch.Generator().manual_seed(8)
    n, v = 16400, 131000
    assert (n - 3) * v > 2 ** 31
    last = (torch.randn(3, v, generator=g) * 3).to(torch.bfloat16)
    z = torch.zeros(n, v, dtype=torch.bfloat16, device="cuda")
    z[-3:] = last.cuda()
    tok = torch.randint(0, v, (n,), generator=g)
    gl, ge = torch.randn(n, generator=g), torch.randn(n, generator=g)
    f = fq.fp4_token_logprobs(z, tok.cuda(), top=2)
    logv = float(torch.log(torch.tensor(v, dtype=F)))
    _near(f.logprob[:-3], torch.full((n - 3,), -logv, dtype=F), "logprob of zeros")
    _near(f.entropy[:-3], torch.full((n - 3,), logv, dtype=F), "entropy of zeros")
    assert (f.top_ids[:-3].cpu() == torch.tensor([0, 1])).all()
    hit, ent, ids, best, *_ = _reference(last, tok[-3:], 1.0, 2)
    _near(f.logprob[-3:], hit, "logprob")
    _near(f.entropy[-3:], ent, "entropy")
    assert torch.equal(f.top_ids[-3:].cpu().long(), ids)
    _near(f.top_logprobs[-3:], best, "top_logprobs")
    dz = fq.fp4_token_logprobs_backward(z, tok.cuda(), f, gl.cuda(), ge.cuda())[-3:].cpu()
    end = fq.fp4_token_logprobs(last.cuda(), tok[-3:].cuda(), top=2)
    want = fq.fp4_token_logprobs_backward(last.cuda(), tok[-3:].cuda(), end, gl[-3:].cuda(), ge[-3:].cuda()).cpu()
    # the two calls may add a row in other pieces: both are within 5e-5 + half a step of the formula's
    assert torch.isclose(dz.float(), want.float(), rtol=2.0 ** -7 + 2e-4, atol=1e-9).all()
    wide = z.flatten().as_strided((3, v), (2 ** 30, 1))
    wide.copy_(last)
    _check(wide, tok[-3:], top=2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temp", [1e-37, 1e-30, 1e-12, 1e30])
@pytest.mark.parametrize("n,v", [(4, 1000), (2, 9000)])
def test_far_temperatures(dtype, temp, n, v):
    """z / temperature may leave binary32 where (z - max) / temperature does
    not matter any more: one token takes all, or all are alike."""
    g = torch.Generator().manual_seed(v)
    z = (torch.randn(n, v, generator=g) * 30).to(dtype)
    z[1] -= 500
    _check(z, _tokens(g, n, v), temp, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v", [(1, 700), (1, 9000), (1, 30011)])
def test_far_logits(dtype, n, v):
    """Rows of masks and rows of large logits, whose distances still matter,
    rising and in any order."""
    g = torch.Generator().manual_seed(v)
    r = torch.randn(v, generator=g)
    rows = [r * 0 - 1e10, r * 0 - 3e12, torch.where(r > 0, -1e10, r), r * 3 + 2e9, r * 1e12, r * 40 - 6.93e7, r * 40 + 6.93e7,
            torch.sort(r).values * 40 - 6.93e7, torch.sort(r).values * 3e7, torch.sort(r.abs()).values * 1e9 - 1e9]
    z = torch.stack(rows).to(dtype)
    for i in range(len(rows)):
        _check(z[i:i + 1], torch.tensor([v // 3]), 1.0, 2)
    _check(z, torch.arange(len(rows)) * 7, 0.25, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v", [(600, 6001), (515, 16383), (2003, 16500), (1999, 16500)])
def test_many_rows(dtype, n, v):
    """Many rows at once: the last ones against binary64, all of them against
    the same rows in small batches, which are cut another way."""
    g = torch.Generator(device="cuda").manual_seed(n + v)
    z = (torch.randn(n, v, generator=g, device="cuda") * 3).to(dtype)
    tok = torch.randint(0, v, (n,), generator=g, device="cuda")
    f = fq.fp4_token_logprobs(z, tok, temperature=0.8, top=20)
    hit, ent, ids, best, *_ = _reference(z[-16:].cpu(), tok[-16:].cpu(), 0.8, 20)
    _near(f.logprob[-16:], hit, "logprob")
    _near(f.entropy[-16:], ent, "entropy")
    assert torch.equal(f.top_ids[-16:].cpu().long(), ids)
    _near(f.top_logprobs[-16:], best, "top_logprobs")
    none = fq.fp4_token_logprobs(z, tok, temperature=0.8)
    for a in range(0, n, 256):
        few = fq.fp4_token_logprobs(z[a:a + 256], tok[a:a + 256], temperature=0.8, top=20)
        assert torch.equal(f.top_ids[a:a + 256], few.top_ids)
        for what in ("logprob", "entropy", "top_logprobs"):        # each within 5e-5 of the formula
            one, two = getattr(f, what)[a:a + 256], getattr(few, what)
            assert ((one - two).abs() <= 1e-4 + two.abs() * 2.0 ** -21).all(), what
        for what in ("logprob", "entropy"):
            one, two = getattr(none, what)[a:a + 256], getattr(few, what)
            assert ((one - two).abs() <= 1e-4 + two.abs() * 2.0 ** -21).all(), what
