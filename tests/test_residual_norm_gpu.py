"""Residual norms (fp4_residual_norm and its backward) against binary64.

Tolerances: a row's sum of squares is a binary32 sum of at most 32 terms a
thread and two tree levels (about 50 roundings, 3e-6 relative at the worst),
so rho is within 3e-6, u and h within 1e-5 of the magnitudes they add, and
each later expression within a few times that of its own magnitudes: 3e-5.
Sums over the rows add at most rows / groups + groups / 4 + 2 further
roundings (below 300 here, 2e-5).  Outputs add half a step of their type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
F = torch.float64
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(rows, cols, xd, rd, wd, post, gate, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, sd=1.0, dtype=FP: (torch.randn(*s, generator=g) * sd).to(dtype)   # noqa: E731
    return dict(x=r(rows, cols, dtype=xd), res=r(rows, cols, sd=2, dtype=rd), w_pre=(1 + r(cols, sd=0.2)).to(wd),
                w_post=(0.5 + r(cols, sd=0.2)).to(wd) if post else None,
                gate=torch.rand(rows, generator=g) * 2 - 0.5 if gate else None,
                dn=r(rows, cols, sd=0.1, dtype=xd), dh=r(rows, cols, sd=0.1, dtype=rd))


def _reference(i, alpha, eps):
    """Outputs and gradients in binary64, each with the magnitude of what it adds."""
    x, res, w2 = i["x"].to(F), i["res"].to(F), i["w_pre"].to(F)
    c = x.shape[1]
    w1 = i["w_post"].to(F) if i["w_post"] is not None else None
    gate = i["gate"].to(F)[:, None] if i["gate"] is not None else torch.ones(len(x), 1, dtype=F)
    r1 = (x.square().mean(-1, keepdim=True) + eps).rsqrt() if w1 is not None else torch.ones(len(x), 1, dtype=F)
    u = x * r1 * w1 if w1 is not None else x
    h = alpha * res + gate * u
    mh = (alpha * res).abs() + (gate * u).abs()
    r2 = (h.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = h * r2 * w2
    mn = mh * r2 * w2.abs() + n.abs()
    out = dict(h=(h, mh), n=(n, mn))
    dn, dh = i["dn"], i["dh"]
    dn = torch.zeros_like(x) if dn is None else dn.to(F)
    dh = torch.zeros_like(x) if dh is None else dh.to(F)
    q = dn * w2
    t = dh + r2 * q - h * r2 ** 3 * (q * h).sum(-1, keepdim=True) / c
    mt = dh.abs() + r2 * q.abs() + mh * r2 ** 3 * (q.abs() * mh).sum(-1, keepdim=True) / c
    out["dres"] = (alpha * t, abs(alpha) * mt)
    out["dw_pre"] = ((dn * h * r2).sum(0), (dn.abs() * mh * r2).sum(0))
    qs, mq = (t * u).sum(-1, keepdim=True), (mt * u.abs()).sum(-1, keepdim=True)
    if i["gate"] is not None:
        out["dgate"] = (qs[:, 0], mq[:, 0])
    if w1 is None:
        out["dx"] = (gate * t, gate.abs() * mt)
    else:
        out["dw_post"] = ((gate * t * x * r1).sum(0), (gate.abs() * mt * x.abs() * r1).sum(0))
        out["dx"] = (r1 * w1 * gate * t - x * r1 ** 2 * gate * qs / c,
                     r1 * w1.abs() * gate.abs() * mt + x.abs() * r1 ** 2 * gate.abs() * mq / c)
    return out


def _close(got, pair, what):
    want, mag = pair
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    off = (got.cpu().to(F) - want).abs()
    tol = (3e-5 + (2e-5 if what.startswith("dw") else 0)) * mag + half * (want.abs() + 1e-4 * mag) + 1e-37
    assert not (~(off <= tol)).any(), (what, float(off.max()), (~(off <= tol)).nonzero()[0].tolist())


def _cuda(i):
    return {k: None if v is None else v.cuda() for k, v in i.items()}


def _run(i, alpha, eps):
    d = _cuda(i)
    kw = dict(w_post=d["w_post"], gate=d["gate"], alpha=alpha)
    h, n, stats = fq.fp4_residual_norm(d["x"], d["res"], d["w_pre"], eps=eps, **kw)
    g = fq.fp4_residual_norm_backward(d["dn"], d["dh"], d["x"], d["res"], d["w_pre"], stats, **kw)
    return dict(h=h, n=n, dx=g.dx, dres=g.dres, dw_pre=g.dw_pre, dw_post=g.dw_post, dgate=g.dgate)


def _check(i, alpha=0.75, eps=1e-6):
    got, want = _run(i, alpha, eps), _reference(i, alpha, eps)
    for k, pair in want.items():
        _close(got[k], pair, k)
    assert got["dw_post"] is None or i["w_post"] is not None
    assert got["dgate"] is None or i["gate"] is not None
    return got


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (2, 8), (5, 64), (130, 513), (3, 520), (700, 1027), (9, 2048),
                                       (4, 2056), (3, 4095), (600, 4096), (2, 5000), (3, 8192), (2, 9001), (2, 16384),
                                       (2, 18944), (2, 32765), (2, 32768)])
@pytest.mark.parametrize("xd,rd,wd", [(BF, BF, BF), (BF, FP, BF), (FP, FP, FP), (FP, BF, FP)])
def test_shapes_and_types(rows, cols, xd, rd, wd):
    _check(_inputs(rows, cols, xd, rd, wd, True, cols % 2 == 1, rows + cols))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("drop", ["", "dn", "dh", "both"])
def test_options(post, gate, drop):
    i = _inputs(37, 1000, BF, FP, FP, post, gate, 5)
    if drop in ("dn", "both"):
        i["dn"] = None
    if drop in ("dh", "both"):
        i["dh"] = None
    _check(i, alpha=-1.5, eps=1e-3)


def test_zero_rows_and_rows_of_other_values():
    """A row of zeros has rho = 1 / sqrt(eps); a NaN or an infinity stays in
    its own row; tiny and large rows keep their precision."""
    i = _inputs(8, 264, FP, FP, FP, True, True, 7)
    i["x"][0], i["res"][0] = 0.0, 0.0
    i["x"][1] *= 1e-12
    i["res"][2] *= 1e6
    i["gate"][3] = 0.0
    got = _check(i)
    bad = dict(i, x=i["x"].clone(), res=i["res"].clone())
    bad["x"][5][3], bad["res"][6][9] = float("nan"), float("inf")
    two = _run(bad, 0.75, 1e-6)
    keep = [0, 1, 2, 3, 4, 7]
    for k in ("h", "n", "dx", "dres", "dgate"):
        assert torch.equal(got[k][keep], two[k][keep]), k
        assert not torch.isfinite(two[k][5].float()).all()


def test_strided_rows():
    """Views of wider tensors, whose rows start at any element: the sums run
    in another order than a dense tensor's, within the same bounds."""
    i = _cuda(_inputs(21, 520, BF, FP, BF, True, True, 3))
    wide = {k: torch.cat([v[:, :8] * 0 + 5, v, v[:, :13] * 0 + 5], 1) for k, v in i.items() if v is not None and v.dim() == 2}
    for cols in (520, 519):
        j = dict(i, **{k: v[:, 8:8 + cols] for k, v in wide.items()})
        j.update({k: j[k][:cols].contiguous() for k in ("w_pre", "w_post")})
        h, n, _, dx, dres, dw2, dw1, dg = _run_cuda(j)
        want = _reference({k: v.cpu() for k, v in j.items()}, 0.5, 1e-6)
        for k, v in dict(h=h, n=n, dx=dx, dres=dres, dw_pre=dw2, dw_post=dw1, dgate=dg).items():
            _close(v, want[k], k)


def _run_cuda(d, stream=None):
    kw = dict(w_post=d["w_post"], gate=d["gate"], alpha=0.5, stream=stream)
    h, n, stats = fq.fp4_residual_norm(d["x"], d["res"], d["w_pre"], **kw)
    g = fq.fp4_residual_norm_backward(d["dn"], d["dh"], d["x"], d["res"], d["w_pre"], stats, **kw)
    return h, n, stats, g.dx, g.dres, g.dw_pre, g.dw_post, g.dgate


def test_gradients_against_differences():
    """<gradient, v> against central differences of the binary64 loss
    sum(dn n + dh h): step 1e-4, truncation of order 1e-8 of third
    derivatives."""
    i = _inputs(5, 96, FP, FP, FP, True, True, 13)
    got = _run(i, 0.75, 1e-6)

    def loss(j):
        r = _reference(j, 0.75, 1e-6)
        return float((i["dn"].to(F) * r["n"][0]).sum() + (i["dh"].to(F) * r["h"][0]).sum())

    g = torch.Generator().manual_seed(1)
    for name, grad in (("x", "dx"), ("res", "dres"), ("w_pre", "dw_pre"), ("w_post", "dw_post"), ("gate", "dgate")):
        v = torch.randn(i[name].shape, generator=g, dtype=F)
        want = (loss(dict(i, **{name: i[name].to(F) + 1e-4 * v})) - loss(dict(i, **{name: i[name].to(F) - 1e-4 * v}))) / 2e-4
        d = got[grad].cpu().to(F)
        assert abs(float((d * v).sum()) - want) <= 1e-4 * float((d.abs() * v.abs()).sum()) + 1e-6, name


def test_empty_batch_streams_and_replay():
    i = _cuda(_inputs(300, 1032, BF, FP, BF, True, True, 2))
    e = {k: v if v is None or k.startswith("w") else v[:0] for k, v in i.items()}
    h, n, stats, dx, dres, dw2, dw1, dg = _run_cuda(e)
    assert h.shape == (0, 1032) and dg.shape == (0,) and (dw2 == 0).all() and (dw1 == 0).all()
    want = [t.clone() for t in _run_cuda(i)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _run_cuda(i, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run_cuda(i)
    for _ in range(4):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(_run_cuda(i), want))
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """More than 2^31 elements: rows of zeros, which give and add zeros, and
    three last rows like any others; then rows far apart in one allocation."""
    rows, cols = 65600, 32768
    assert (rows - 3) * cols > 2 ** 31
    i = _inputs(3, cols, BF, BF, BF, True, True, 21)
    d = _cuda(i)
    for k in ("x", "res", "dn", "dh"):
        v = torch.zeros(rows, cols, dtype=BF, device="cuda")
        v[-3:] = d[k]
        d[k] = v
    d["gate"] = torch.cat([torch.ones(rows - 3, device="cuda"), d["gate"]])
    h, n, _, dx, dres, dw2, dw1, dg = _run_cuda(d)
    want = _reference(i, 0.5, 1e-6)
    for k, v in dict(h=h, n=n, dx=dx, dres=dres).items():
        assert not v[:-3].any(), k
        _close(v[-3:], want[k], k)
    for k, v in dict(dw_pre=dw2, dw_post=dw1, dgate=dg[-3:]).items():
        _close(v, want[k], k)
    j = dict(_cuda(i), gate=d["gate"][-3:])
    for k in ("x", "res", "dn", "dh"):
        j[k] = d[k].flatten().as_strided((3, cols), (2 ** 30, 1))
        j[k].copy_(i[k])
    h, n, _, dx, dres, dw2, dw1, dg = _run_cuda(j)
    for k, v in dict(h=h, n=n, dx=dx, dres=dres, dw_pre=dw2, dw_post=dw1, dgate=dg).items():
        _close(v, want[k], k)
