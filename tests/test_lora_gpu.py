"""Low-rank adapters (fp4_lora_apply, fp4_lora_backward, fp4_wo_gemm_lora)
against binary64.

Tolerances: every product of two bf16 values is exact in binary32, and the
library's products are held to 1e-5 of the sum of their terms' magnitudes.
A value that enters a second product as hi + lo bf16 terms is off by at most
2^-17 < 1e-5 of itself.  So a result of two chained products is within 3e-5
of the sum of magnitudes through both (1e-5 each, and the split), plus half a
step of the output's type (bf16 2^-8 relative, fp32 2^-24)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
F = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _randn(g, *shape, sd=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * sd).to(dtype)


def _slots(g, m, la, how):
    if how == "none":
        return torch.full((m,), -1, dtype=torch.int32)
    if how == "one":
        return torch.full((m,), la - 1, dtype=torch.int32)
    if how == "mixed":                                    # any order, rows outside the bank among them
        s = torch.randint(-1, la + 1, (m,), generator=g)
        if m > 2:
            s[m // 2] = -2147483648
            s[m // 3] = 2147483647
        return s.to(torch.int32)
    cuts = torch.randint(0, m + 1, (4,), generator=g).sort().values
    run = torch.bucketize(torch.arange(m), cuts, right=True)
    return torch.tensor([0, -1, la - 1, la // 2, 0], dtype=torch.int32)[run]


def _bank(g, la, n, k, r):
    return _randn(g, la, r, k, sd=k ** -0.5), _randn(g, la, n, r, sd=0.1), torch.rand(la, generator=g) + 0.5


def _dev(*ts):
    return [t.cuda() for t in ts]


def _rows_of(slots, i):
    return (slots == i).nonzero()[:, 0]


def _forward64(x, a, b, scale, slots, base):
    """(y, t, magnitude of the adapter's sums, magnitude of t's)."""
    m, (la, n, r) = x.shape[0], b.shape
    y = torch.zeros(m, n, dtype=F) if base is None else base.to(F).clone()
    t, my, mt = torch.zeros(m, r, dtype=F), torch.zeros(m, n, dtype=F), torch.zeros(m, r, dtype=F)
    for i in range(la):
        at = _rows_of(slots, i)
        ai, bi, s = a[i].to(F), b[i].to(F), float(scale[i])
        t[at] = x[at].to(F) @ ai.t()
        mt[at] = x[at].to(F).abs() @ ai.abs().t()
        y[at] += s * (t[at] @ bi.t())
        my[at] = s * (mt[at] @ bi.abs().t())
    return y, t, my, mt


def _close(got, want, mag, rel, dtype, what):
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype] / 1.0
    tol = rel * mag + half * (want.abs() + rel * mag)
    off = (got.cpu().to(F) - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(off[bad].max()))


SHAPES = [  # m, n, k, rank, adapters, slots
    (1, 8, 8, 8, 1, "one"), (1, 520, 264, 16, 3, "one"), (2, 72, 1000, 24, 2, "mixed"), (3, 264, 40, 128, 4, "mixed"),
    (16, 1000, 520, 32, 16, "mixed"), (17, 256, 256, 8, 2, "runs"), (33, 40, 2056, 72, 5, "mixed"),
    (63, 248, 136, 40, 2, "none"), (64, 264, 384, 64, 1, "one"), (65, 512, 200, 16, 3, "runs"),
    (130, 264, 520, 8, 3, "runs"), (200, 1032, 4096, 32, 2, "mixed"), (300, 776, 776, 128, 3, "runs"),
    (2100, 1032, 136, 16, 3, "runs"), (2050, 520, 264, 24, 2, "mixed"), (3000, 776, 136, 32, 40, "mixed"),
    (2048, 512, 40, 8, 1, "none"), (2500, 600, 72, 16, 1, "one"),
    (1100, 264, 3848, 16, 4, "runs"), (2050, 72, 2104, 40, 3, "mixed"), (600, 136, 7208, 128, 2, "runs"), (4200, 520, 1032, 24, 5, "runs"),
    (530, 136, 8200, 72, 2, "one"), (9, 520, 264, 96, 3, "mixed"),
    (513, 136, 264, 56, 40, "mixed"), (1100, 264, 392, 16, 4, "runs"), (2050, 264, 136, 48, 2, "mixed"),
]


@pytest.mark.parametrize("m,n,k,r,la,how", SHAPES)
@pytest.mark.parametrize("base", [False, True])
def test_apply(m, n, k, r, la, how, base):
    g = torch.Generator().manual_seed(m * 7 + n + k + r)
    x, (a, b, sc) = _randn(g, m, k), _bank(g, la, n, k, r)
    slots, bs = _slots(g, m, la, how), _randn(g, m, n) if base else None
    xd, ad, bd, sd, sl = _dev(x, a, b, sc, slots)
    y, t = fq.fp4_lora_apply(xd, fq.LoraBank(ad, bd, sd), sl, base=None if bs is None else bs.cuda())
    y64, t64, my, mt = _forward64(x, a, b, sc, slots, bs)
    _close(t, t64, mt, 1e-5, torch.float32, "t")
    _close(y, y64, my, 3e-5, torch.bfloat16, "y")
    out = ~((slots >= 0) & (slots < la))
    assert (t.cpu()[out] == 0).all()
    assert torch.equal(y.cpu()[out], bs[out] if base else torch.zeros(int(out.sum()), n, dtype=torch.bfloat16))


def _backward64(dy, x, t, a, b, sc, slots, dxb):
    z = torch.zeros
    dx = z(x.shape, dtype=F) if dxb is None else dxb.to(F).clone()
    mdx, da, mda = z(x.shape, dtype=F), z(a.shape, dtype=F), z(a.shape, dtype=F)
    db, mdb = z(b.shape, dtype=F), z(b.shape, dtype=F)
    for i in range(a.shape[0]):
        at = _rows_of(slots, i)
        ai, bi, s = a[i].to(F), b[i].to(F), float(sc[i])
        d, xi, ti = dy[at].to(F), x[at].to(F), t[at].to(F)
        dt, mdt = s * (d @ bi), s * (d.abs() @ bi.abs())
        dx[at] += dt @ ai
        mdx[at] = mdt @ ai.abs()
        da[i], mda[i] = dt.t() @ xi, mdt.t() @ xi.abs()
        db[i], mdb[i] = s * (d.t() @ ti), s * (d.abs().t() @ ti.abs())
    return dx, da, db, mdx, mda, mdb


@pytest.mark.parametrize("m,n,k,r,la,how", SHAPES)
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
def test_backward(m, n, k, r, la, how, gdt):
    g = torch.Generator().manual_seed(m * 11 + n + k + r)
    x, dy, (a, b, sc) = _randn(g, m, k), _randn(g, m, n, sd=0.1), _bank(g, la, n, k, r)
    slots = _slots(g, m, la, how)
    t = _forward64(x, a, b, sc, slots, None)[1].float()
    dxb = _randn(g, m, k) if (m + r) % 3 else None
    xd, dyd, td, ad, bd, sd, sl = _dev(x, dy, t, a, b, sc, slots)
    dx, da, db = fq.fp4_lora_backward(dyd, xd, td, fq.LoraBank(ad, bd, sd), sl,
                                      dx_base=None if dxb is None else dxb.cuda(), grad_dtype=gdt)
    dx64, da64, db64, mdx, mda, mdb = _backward64(dy, x, t, a, b, sc, slots, dxb)
    _close(dx, dx64, mdx, 3e-5, torch.bfloat16, "dx")
    _close(da, da64, mda, 3e-5, gdt, "da")
    _close(db, db64, mdb, 3e-5, gdt, "db")
    again = fq.fp4_lora_backward(dyd, xd, td, fq.LoraBank(ad, bd, sd), sl,
                                 dx_base=None if dxb is None else dxb.cuda(), grad_dtype=gdt)
    for one, two in zip((dx, da, db), again):              # sums in a fixed order
        assert torch.equal(one, two)


def test_backward_against_differences():
    """<gradient, v> against (f(p + h v) - f(p - h v)) / 2h of the binary64
    loss sum(dy y).  The loss is linear in each of x, A and B, so the central
    difference is exact but for binary64 rounding."""
    g = torch.Generator().manual_seed(5)
    m, n, k, r, la = 70, 136, 264, 16, 3
    x, dy, (a, b, sc) = _randn(g, m, k), _randn(g, m, n, sd=0.1), _bank(g, la, n, k, r)
    slots = _slots(g, m, la, "mixed")
    y64, t64, _, _ = _forward64(x, a, b, sc, slots, None)
    xd, dyd, td, ad, bd, sd, sl = _dev(x, dy, t64.float(), a, b, sc, slots)
    got = fq.fp4_lora_backward(dyd, xd, td, fq.LoraBank(ad, bd, sd), sl)
    mags = _backward64(dy, x, t64, a, b, sc, slots, None)[3:]
    for i, p in enumerate((x, a, b)):
        v = torch.randn(p.shape, generator=g, dtype=F)
        loss = []
        for h in (1e-3, -1e-3):
            q = [x.to(F), a.to(F), b.to(F)]
            q[i] = q[i] + h * v
            loss.append(float((dy.to(F) * _forward64(*q, sc, slots, None)[0]).sum()))
        want = (loss[0] - loss[1]) / 2e-3
        dot = float((got[i].cpu().to(F) * v).sum())
        half = 2.0 ** -8 if i == 0 else 2.0 ** -24         # dx leaves in bf16, da and db in fp32
        tol = float(((3e-5 + half) * mags[i] * v.abs()).sum()) + 1e-9
        assert abs(dot - want) <= tol, (i, dot, want, tol)


def test_rows_without_an_adapter_stay_out_of_everything():
    """NaN and infinities in rows without an adapter, in another adapter's
    rows and in an unused adapter reach nothing else; in place, such rows keep
    their bits."""
    g = torch.Generator().manual_seed(9)
    m, n, k, r, la = 100, 264, 136, 16, 4
    x, dy, (a, b, sc) = _randn(g, m, k), _randn(g, m, n, sd=0.1), _bank(g, la, n, k, r)
    slots = torch.randint(0, 2, (m,), generator=g, dtype=torch.int32)
    slots[::7] = -1
    slots[5::7] = 2
    clean = slots < 2
    bad = ~clean
    bs = _randn(g, m, n)
    xb, dyb, ab, bb = x.clone(), dy.clone(), a.clone(), b.clone()
    xb[bad], dyb[bad] = float("nan"), float("inf")
    ab[2:], bb[3] = float("nan"), float("-inf")
    tb = torch.randn(m, r, generator=g)
    tb[bad] = float("nan")
    td = tb.clone()
    td[bad] = 0.0
    res = []
    for xs, ds, as_, bs_, ts in ((x, dy, a, b, td), (xb, dyb, ab, bb, tb)):
        xd, dd, ad, bd, sd, sl, tdv = _dev(xs, ds, as_, bs_, sc, slots, ts)
        bank = fq.LoraBank(ad, bd, sd)
        y = bs.cuda()
        y, t = fq.fp4_lora_apply(xd, bank, sl, base=y, out=y)
        dx, da, db = fq.fp4_lora_backward(dd, xd, tdv, bank, sl)
        res.append((y.cpu(), t.cpu(), dx.cpu(), da.cpu(), db.cpu()))
    one, two = res
    for i in (0, 1, 2):
        assert torch.equal(one[i][clean], two[i][clean]), i
    none = slots < 0
    assert torch.equal(two[0][none], bs[none]) and (two[1][none] == 0).all() and (two[2][none] == 0).all()
    for i in (3, 4):
        assert torch.equal(one[i][:2], two[i][:2]), i
        assert (two[i][3] == 0).all()                      # an adapter without rows


def test_strided_rows_and_empty_batches():
    g = torch.Generator().manual_seed(3)
    m, n, k, r, la = 37, 136, 264, 24, 2
    x, dy, (a, b, sc) = _randn(g, m, k + 16), _randn(g, m, n + 8), _bank(g, la, n, k, r)
    slots = _slots(g, m, la, "mixed")
    xd, dyd, ad, bd, sd, sl = _dev(x, dy, a, b, sc, slots)
    bank = fq.LoraBank(ad, bd, sd)
    wide = torch.full((m, n + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    y, t = fq.fp4_lora_apply(xd[:, 8:8 + k], bank, sl, base=dyd[:, :n], out=wide[:, 8:8 + n])
    y2, t2 = fq.fp4_lora_apply(xd[:, 8:8 + k].contiguous(), bank, sl, base=dyd[:, :n].contiguous())
    assert torch.equal(y, y2) and torch.equal(t, t2)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + n:] == 7).all()
    g1 = fq.fp4_lora_backward(dyd[:, :n], xd[:, 8:8 + k], t, bank, sl)
    g2 = fq.fp4_lora_backward(dyd[:, :n].contiguous(), xd[:, 8:8 + k].contiguous(), t, bank, sl)
    for u, v in zip(g1, g2):
        assert torch.equal(u, v)
    none = torch.empty(0, k, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    y, t = fq.fp4_lora_apply(none, bank, e)
    assert y.shape == (0, n) and t.shape == (0, r)
    dx, da, db = fq.fp4_lora_backward(y, none, t, bank, e)
    assert dx.shape == (0, k) and (da == 0).all() and (db == 0).all()


# ---------------------------------------------------------------------------
def _dequant64(q):
    return fq.fp4_dequantize(q, torch.float32).cpu().to(F)


WO = [  # m, n, k, rank, adapters, slots, block, scale, element
    (1, 48, 256, 8, 1, "one", 16, "e4m3", "e2m1"), (1, 8208, 512, 16, 4, "one", 16, "e4m3", "e2m1"),
    (3, 1000, 1024, 32, 3, "mixed", 32, "e8m0", "e2m1"), (4, 8200, 256, 128, 2, "mixed", 16, "ue5m3", "e2m1"),
    (5, 77, 2048, 24, 2, "mixed", 16, "e4m3", "e2m1"), (8, 9001, 512, 16, 9, "mixed", 16, "e4m3", "int4"),
    (13, 515, 3584, 64, 5, "mixed", 16, "e3m4", "e2m1"), (16, 8209, 512, 16, 16, "mixed", 16, "e4m3", "e2m1"),
    (16, 264, 2560, 128, 16, "mixed", 32, "e8m0", "fp8_e4m3"), (9, 130, 512, 40, 3, "mixed", 32, "e8m0", "fp6_e2m3"),
    (16, 100, 256, 16, 2, "none", 16, "e4m3", "e2m1"), (2, 96, 256, 8, 2, "runs", 32, "e8m0", "int8"),
]


@pytest.mark.parametrize("m,n,k,r,la,how,block,scale,elem", WO)
def test_weight_only_product_with_adapters(m, n, k, r, la, how, block, scale, elem):
    g = torch.Generator().manual_seed(m + n + k + r)
    x, (a, b, sc) = _randn(g, m, k), _bank(g, la, n, k, r)
    slots = _slots(g, m, la, how)
    w = _randn(g, n, k, sd=0.05).cuda()
    q = fq.fp4_quantize(w, block, scale, amax="none" if scale == "e8m0" else "current", element=elem)
    xd, ad, bd, sd, sl = _dev(x, a, b, sc, slots)
    y = fq.fp4_wo_gemm_lora(xd, q, fq.LoraBank(ad, bd, sd), sl)
    w64 = _dequant64(q)
    y64, _, my, _ = _forward64(x, a, b, sc, slots, x.to(F) @ w64.t())
    _close(y, y64, my + x.to(F).abs() @ w64.abs().t(), 3e-5, torch.bfloat16, "y")
    plain = fq.fp4_wo_gemm(xd, q)
    out = ~((slots >= 0) & (slots < la))
    assert torch.equal(y.cpu()[out], plain.cpu()[out])     # no adapter: the product's own bits


def test_side_stream_and_graph_replay():
    """On another stream than the current one, and captured: every replay
    gives the eager call's bits, with eager work between the replays."""
    g = torch.Generator().manual_seed(21)
    m, n, k, r, la = 300, 520, 1032, 16, 3
    x, dy, (a, b, sc) = _randn(g, m, k), _randn(g, m, n, sd=0.1), _bank(g, la, n, k, r)
    xd, dyd, ad, bd, sd, sl = _dev(x, dy, a, b, sc, _slots(g, m, la, "mixed"))
    bank = fq.LoraBank(ad, bd, sd)

    def step(stream=None):
        y, t = fq.fp4_lora_apply(xd, bank, sl, base=dyd, stream=stream)
        return (y, t, *fq.fp4_lora_backward(dyd, xd, t, bank, sl, stream=stream))

    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        got = step(st)
        side.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        for v in got:
            v.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v)
        for u, v in zip(step(), want):
            assert torch.equal(u, v)
        torch.cuda.synchronize()


@pytest.mark.parametrize("m", [4, 20])
def test_offsets_past_32_bits(m):
    """Rows far apart in one large allocation, and a bank of more than 2^31
    elements: the last rows and the last adapters are the ones in use."""
    g = torch.Generator().manual_seed(m)
    la, n, k, r = 16384, 1032, 256, 128
    assert la * n * r > 2 ** 31
    x, dy = _randn(g, m, k), _randn(g, m, n)
    some = {la - 1: 0, 3: 1, la - 9: 2}
    a, b, sc = _bank(g, 3, n, k, r)
    ad = torch.zeros(la, r, k, dtype=torch.bfloat16, device="cuda")
    bd = torch.zeros(la, n, r, dtype=torch.bfloat16, device="cuda")
    sd = torch.ones(la, device="cuda")
    for at, i in some.items():
        ad[at], bd[at], sd[at] = a[i].cuda(), b[i].cuda(), sc[i].cuda()
    few = torch.randint(-1, 3, (m,), generator=g).to(torch.int32)
    few[:4] = torch.tensor([0, 1, 2, -1])
    slots = torch.full((m,), -1, dtype=torch.int32)
    for at, i in some.items():
        slots[few == i] = at
    far = (2 ** 31 + 2 ** 26) // (m - 1) // 8 * 8
    assert far * (m - 1) > 2 ** 31

    def spread(v):
        w = torch.empty(far * (m - 1) + v.shape[1], dtype=torch.bfloat16, device="cuda").as_strided((m, v.shape[1]), (far, 1))
        w.copy_(v)
        return w

    bank, sl = fq.LoraBank(ad, bd, sd), slots.cuda()
    xd, dyd = spread(x), spread(dy)
    y, t = fq.fp4_lora_apply(xd, bank, sl, base=dyd, out=spread(torch.zeros_like(dy)))
    y64, t64, my, mt = _forward64(x, a, b, sc, few, dy)
    _close(t, t64, mt, 1e-5, torch.float32, "t")
    _close(y, y64, my + dy.to(F).abs(), 3e-5, torch.bfloat16, "y")
    dx, da, db = fq.fp4_lora_backward(dyd, xd, t, bank, sl)
    dx64, da64, db64, mdx, mda, mdb = _backward64(dy, x, t.cpu(), a, b, sc, few, None)
    _close(dx, dx64, mdx, 3e-5, torch.bfloat16, "dx")
    used, which = torch.tensor(list(some), device="cuda"), list(some.values())
    rest = torch.ones(la, dtype=torch.bool, device="cuda")
    rest[used] = False
    for got, want, mag, what in ((da, da64, mda, "da"), (db, db64, mdb, "db")):
        assert not got.flatten(1).any(1)[rest].any(), what
        _close(got[used], want[which], mag[which], 3e-5, torch.float32, what)
    if m <= 16:
        q = fq.fp4_quantize(_randn(g, n, k, sd=0.05).cuda(), 16, "e4m3", amax="current")
        y = fq.fp4_wo_gemm_lora(x.cuda(), q, bank, sl)
        w64 = _dequant64(q)
        y64, _, my, _ = _forward64(x, a, b, sc, few, x.to(F) @ w64.t())
        _close(y, y64, my + x.to(F).abs() @ w64.abs().t(), 3e-5, torch.bfloat16, "wo y")
