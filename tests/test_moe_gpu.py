"""The mixture-of-experts layer and its router's choice against binary64.

Tolerances of the layer.  A product's sums are within 1e-5 sum |x||w| of the
exact ones (include/fp4.h's bound for the products).  act's slope is below
1.13 and its value within (|g| + 8) 2^-22 of itself.  What it gives enters the
down projection as two bf16 terms, 2^-15 of itself at most off; y is rounded
once, 2^-8."""
import math

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq
from tests.test_epilogue_gpu import act64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def bank_of(experts, hidden, ffn, seed, block=16, scale="e4m3", element="e2m1", down=None, each=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(rows, cols, fmt):
        b, s, e = fmt
        w = torch.randn(experts * rows, cols, generator=g, device="cuda") * 0.1
        return fq.fp4_quantize(w.to(BF), b, s, amax="none" if s == "e8m0" else "current", element=e)
    fmt = (block, scale, element)
    sc = [torch.rand(experts, generator=g, device="cuda") + 0.5 for _ in range(2)] if each else [None, None]
    return fq.MoeBank(make(2 * ffn, hidden, fmt), make(hidden, ffn, down or fmt), experts, *sc)


def layer64(x, bank, ids, weights, act, residual):
    """(y, error bound before the last rounding)."""
    E, h, f = bank.experts, bank.gate_up.cols, bank.down.cols
    up = fq.fp4_dequantize(bank.gate_up).double().view(E, 2 * f, h)
    down = fq.fp4_dequantize(bank.down).double().view(E, h, f)
    if bank.up_scale is not None:
        up = up * bank.up_scale.double()[:, None, None]
        down = down * bank.down_scale.double()[:, None, None]
    x64 = x.double()
    y = torch.zeros_like(x64) if residual is None else residual.double()
    err = 2.0 ** -22 * y.abs()
    for m in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e, w = int(ids[m, k]), float(weights[m, k])
            if not 0 <= e < E:
                continue
            s, es = up[e] @ x64[m], 1e-5 * (up[e].abs() @ x64[m].abs())
            g, u = s[:f], s[f:]
            a = act64(g, act)
            hh = a * u
            eh = u.abs() * (1.13 * es[:f] + (g.abs() + 8.0) * 2.0 ** -22 * a.abs()) + a.abs() * es[f:] + 2.0 ** -15 * hh.abs()
            y[m] += w * (down[e] @ hh)
            err[m] += abs(w) * (down[e].abs() @ (1.01 * eh + 1e-5 * hh.abs()))
    return y, err


def check(y, x, bank, ids, weights, act="silu", residual=None):
    want, err = layer64(x, bank, ids.cpu(), weights.cpu(), act, residual)
    bad = (y.double() - want).abs() > err + 2.0 ** -8 * want.abs() + 1e-37
    assert not bad.any(), (int(bad.sum()), (y.double() - want).abs().max().item())


def choice(m, experts, top, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return fq.fp4_moe_route(torch.randn(m, experts, generator=g, device="cuda"), top)


def tokens(m, h, seed):
    return torch.randn(m, h, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(BF)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 13, 16])
@pytest.mark.parametrize("experts,top", [(1, 1), (5, 2), (40, 8)])
def test_layer(m, experts, top):
    bank = bank_of(experts, 256, 384, m + experts)
    x = tokens(m, 256, m)
    ids, w = choice(m, experts, top, m)
    r = tokens(m, 256, 99)
    check(fq.fp4_moe(x, bank, ids, w, residual=r), x, bank, ids, w, residual=r)
    check(fq.fp4_moe(x, bank, ids, w, act="gelu"), x, bank, ids, w, "gelu")


@pytest.mark.parametrize("hidden,ffn", [(128, 128), (128, 640), (640, 128), (2048, 768), (1152, 896)])
@pytest.mark.parametrize("m", [1, 6, 16])
def test_layer_sizes(hidden, ffn, m):
    bank = bank_of(6, hidden, ffn, hidden + ffn, each=False)
    x = tokens(m, hidden, m)
    ids, w = choice(m, 6, 3, m)
    check(fq.fp4_moe(x, bank, ids, w, act="relu"), x, bank, ids, w, "relu")


@pytest.mark.parametrize("block,scale,element", [
    (32, "e8m0", "e2m1"), (16, "e8m0", "e2m1"), (32, "e4m3", "e2m1"), (16, "ue5m3", "e2m1"), (16, "e1m6", "e2m1"),
    (32, "e8m0", "int4"), (16, "e2m5", "int4"), (32, "e8m0", "fp8_e4m3"), (16, "e4m3", "fp8_e4m3"), (32, "e8m0", "int8"),
    (16, "e4m3", "int8"), (32, "e8m0", "fp6_e2m3"), (16, "e4m3", "fp6_e2m3"), (32, "e8m0", "fp6_e3m2"), (32, "e8m0", "int6"),
    (16, "e4m3", "int6")])
@pytest.mark.parametrize("m", [1, 3, 7, 16])
def test_layer_grids(block, scale, element, m):
    bank = bank_of(4, 256, 256, 5, block, scale, element)
    x = tokens(m, 256, m)
    ids, w = choice(m, 4, 2, m + 1)
    check(fq.fp4_moe(x, bank, ids, w), x, bank, ids, w)


def test_layer_of_two_grids():
    bank = bank_of(3, 256, 384, 6, 16, "e4m3", "e2m1", down=(32, "e8m0", "fp8_e4m3"))
    x = tokens(5, 256, 7)
    ids, w = choice(5, 3, 2, 8)
    check(fq.fp4_moe(x, bank, ids, w, act="gelu_tanh"), x, bank, ids, w, "gelu_tanh")


def test_all_tokens_on_one_expert_and_none():
    bank = bank_of(9, 256, 256, 11)
    x, r = tokens(16, 256, 12), tokens(16, 256, 13)
    ids = torch.full((16, 2), 7, dtype=torch.int32, device="cuda")
    ids[:, 1] = -1
    ids[5] = torch.tensor([-1, 900])                        # no expert at all
    w = torch.rand(16, 2, device="cuda")
    y = fq.fp4_moe(x, bank, ids, w, residual=r)
    check(y, x, bank, ids, w, residual=r)
    assert torch.equal(y[5], r[5])
    none = torch.full((16, 16), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(fq.fp4_moe(x, bank, none, torch.ones(16, 16, device="cuda")), torch.zeros_like(x))


@pytest.mark.parametrize("m,experts,top", [(16, 16, 16), (16, 17, 16), (13, 16, 15), (4, 16, 16), (1, 16, 16), (9, 3, 3)])
def test_every_token_on_nearly_every_expert(m, experts, top):
    """Many tokens on each of many experts, in another order for each token."""
    bank = bank_of(experts, 256, 256, 31)
    x = tokens(m, 256, 32)
    g = torch.Generator(device="cuda").manual_seed(33)
    ids = torch.stack([torch.randperm(experts, generator=g, device="cuda")[:top] for _ in range(m)]).to(torch.int32).contiguous()
    w = torch.rand(m, top, generator=g, device="cuda")
    check(fq.fp4_moe(x, bank, ids, w), x, bank, ids, w)


def test_the_same_expert_twice():
    bank = bank_of(4, 256, 256, 14)
    x = tokens(3, 256, 15)
    ids = torch.tensor([[2, 2, 1], [0, 3, 0], [1, 1, 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.25, 0.5, 1.0], [1.0, -0.5, 2.0], [0.5, 0.25, 0.25]], device="cuda")
    check(fq.fp4_moe(x, bank, ids, w), x, bank, ids, w)


def test_sixteen_choices_of_sixteen_tokens():
    """256 pairs: as many as a call can hold, each with an expert of its own."""
    bank = bank_of(256, 128, 128, 16)
    x = tokens(16, 128, 17)
    ids = torch.randperm(256, device="cuda").to(torch.int32).view(16, 16).contiguous()
    w = torch.rand(16, 16, device="cuda")
    check(fq.fp4_moe(x, bank, ids, w), x, bank, ids, w)


def test_nothing_crosses_tokens_or_experts():
    """A NaN token, and an expert whose scales are NaN, reach only the tokens that have them."""
    bank = bank_of(4, 256, 256, 18)
    x = tokens(6, 256, 19)
    ids = torch.tensor([[0, 1], [1, 2], [0, 2], [3, 0], [1, 0], [2, 3]], dtype=torch.int32, device="cuda")
    w = torch.rand(6, 2, device="cuda")
    clean = fq.fp4_moe(x, bank, ids, w)
    bad = x.clone()
    bad[2, 5] = float("nan")
    y = fq.fp4_moe(bad, bank, ids, w)
    assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3, 4, 5]], clean[[0, 1, 3, 4, 5]])
    bank.down.scales[3 * 256:] = 0x7F                       # expert 3
    y = fq.fp4_moe(x, bank, ids, w)
    assert torch.isnan(y[[3, 5]]).all() and torch.equal(y[[0, 1, 2, 4]], clean[[0, 1, 2, 4]])


def test_an_infinity_stays_one():
    """A weight-one expert, so that only the infinite product is not finite."""
    bank = bank_of(1, 128, 128, 20, each=False)
    x = torch.full((1, 128), 3e38, device="cuda").to(BF)
    ids, w = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    y = fq.fp4_moe(x, bank, ids, w, act="none")
    assert not torch.isfinite(y).any()


def positive_bank(seed, block, scale, element, sign):
    """One expert whose codes are all of one sign in each matrix, none of them zero: gate and up positive, down `sign`."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(rows, s):
        w = s * (torch.rand(rows, 256, generator=g, device="cuda") * 0.5 + 0.5)
        q = fq.fp4_quantize(w.to(BF), block, scale, amax="none" if scale == "e8m0" else "current", element=element)
        assert (s * fq.fp4_dequantize(q) > 0).all()
        return q
    return fq.MoeBank(make(512, 1.0), make(256, sign), 1)


# in the last six a weight enters as two terms, of which the second may be zero
@pytest.mark.parametrize("block,scale,element", [
    (16, "e4m3", "e2m1"), (32, "e8m0", "e2m1"), (32, "e8m0", "fp8_e4m3"), (32, "e8m0", "int8"), (32, "e8m0", "fp6_e3m2"),
    (16, "e1m6", "e2m1"), (16, "e2m5", "int4"), (16, "ue5m3", "int8"), (16, "e4m3", "int8"), (32, "e4m3", "int6"),
    (16, "e1m6", "fp8_e4m3")])
@pytest.mark.parametrize("m", [1, 3, 16])
def test_an_infinity_keeps_its_sign(m, block, scale, element):
    """Weights of one sign: an infinity that act gives, or that x holds, reaches y as one and never as a NaN."""
    ids, w = torch.zeros(m, 1, dtype=torch.int32, device="cuda"), torch.ones(m, 1, device="cuda")
    for sign in (1.0, -1.0):
        bank = positive_bank(28, block, scale, element, sign)
        x = torch.full((m, 256), 3e38, device="cuda").to(BF)     # finite: the products overflow
        y = fq.fp4_moe(x, bank, ids, w)
        assert (y == sign * math.inf).all()
        x = torch.rand(m, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(29)).to(BF)
        x[0, 77] = math.inf
        y = fq.fp4_moe(x, bank, ids, w)
        assert (y[0] == sign * math.inf).all() and torch.isfinite(y[1:]).all()


def picking_bank(scale):
    """Two experts whose down projection is the identity: the first gives scale^2 x[0] x[64] everywhere, the second x[127]^2."""
    gate, up = torch.zeros(2, 128, 128, device="cuda"), torch.zeros(2, 128, 128, device="cuda")
    gate[0, :, 0], up[0, :, 64], gate[1, :, 127], up[1, :, 127] = 1.0, 1.0, 1.0, 1.0
    one = [fq.fp4_quantize(w.to(BF), 32, "e8m0", amax="none") for w in (
        torch.cat([gate, up], 1).view(512, 128), torch.eye(128, device="cuda").repeat(2, 1))]
    return fq.MoeBank(*one, 2, torch.tensor([scale, 1.0], device="cuda"))


def test_the_hidden_value_has_seventeen_bits():
    """The first expert's hidden value h, less h64 by the second's router weight: what is left is the rounding of h to
    its two terms.  Both to nearest: the first is off by at most 2^-8 of h's binade, so that the second's last place is
    2^-16 of it, and half of that, 2^-17, is the error at most.  Before it the two scales, act's product and h64 in
    binary32, 4 2^-24 of h; after it y's rounding, 2^-8 of what is left."""
    g = torch.Generator(device="cuda").manual_seed(30)
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(16, 1)
    worst = 0.0
    for _ in range(40):
        scale = float(torch.rand(1, generator=g, device="cuda") + 1.0)
        x = torch.zeros(16, 128, device="cuda")
        x[:, 0], x[:, 64] = torch.rand(2, 16, generator=g, device="cuda") + 0.5
        x[:, 127] = 1.0
        x = x.to(BF)
        h = x[:, 0].double() * x[:, 64].double() * float(torch.tensor(scale)) ** 2
        w = torch.stack([torch.ones(16, device="cuda"), -h.float()], 1).contiguous()
        y = fq.fp4_moe(x, picking_bank(scale), ids, w, act="none").double()
        binade = torch.exp2(torch.floor(torch.log2(h)))
        off = (y.abs() * (1 - 2.0 ** -8) - 2.0 ** -22 * h[:, None]) / binade[:, None]
        worst = max(worst, off.max().item())
    assert worst <= 2.0 ** -17


def test_a_hidden_value_past_bf16_is_finite():
    """binary32 reaches 2^-8 further than bf16: a hidden value there is no infinity."""
    x = torch.zeros(1, 128, device="cuda")
    x[0, 0], x[0, 64], x[0, 127] = torch.finfo(BF).max, 1.0, 1.0
    scale = 1.0015
    h = torch.finfo(BF).max * float(torch.tensor(scale)) ** 2
    assert torch.finfo(BF).max < h < torch.finfo(torch.float32).max
    ids, w = torch.tensor([[0]], dtype=torch.int32, device="cuda"), torch.tensor([[0.5]], device="cuda")
    y = fq.fp4_moe(x.to(BF), picking_bank(scale), ids, w, act="none").double()
    assert ((y - 0.5 * h).abs() <= (2.0 ** -8 + 2.0 ** -15) * 0.5 * h).all()


def test_strided_rows_and_in_place():
    bank = bank_of(5, 256, 256, 21)
    wide = tokens(7, 264, 22)
    x = wide[:, :256]
    ids, w = choice(7, 5, 2, 23)
    r = tokens(7, 259, 24)
    keep = r.clone()
    y = fq.fp4_moe(x, bank, ids, w, residual=r[:, :256], out=r[:, :256])
    check(y, x, bank, ids, w, residual=keep[:, :256])
    assert torch.equal(r[:, 256:], keep[:, 256:])
    z = x.contiguous()
    want = fq.fp4_moe(z, bank, ids, w, residual=z)
    fq.fp4_moe(z, bank, ids, w, residual=z, out=z)
    assert torch.equal(z, want)


def test_layer_bits_repeat():
    bank = bank_of(30, 512, 512, 25)
    x = tokens(16, 512, 26)
    ids, w = choice(16, 30, 6, 27)
    y = fq.fp4_moe(x, bank, ids, w)
    for _ in range(4):
        assert torch.equal(fq.fp4_moe(x, bank, ids, w), y)


# ---------------------------------------------------------------------------
def route64(z, top, score, bias, renormalize, scale):
    z = z.double()
    s = torch.softmax(z, -1) if score == "softmax" else torch.sigmoid(z)
    by = (z if bias is None else s + bias.double()).masked_fill(z == -math.inf, -math.inf)
    ids = torch.argsort(by, dim=-1, descending=True, stable=True)[:, :top]
    p = s.gather(1, ids)
    gone = z.gather(1, ids) == -math.inf
    p = torch.where(gone, 0.0, p)
    if renormalize:
        t = p.sum(-1, keepdim=True)
        p = torch.where(t == 0, 0.0, p / t)
    return torch.where(gone, -1, ids).to(torch.int32), scale * p


@pytest.mark.parametrize("rows,experts", [(1, 1), (1, 8), (3, 64), (16, 65), (5, 127), (33, 256), (9, 1000), (700, 40), (2, 1024)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(rows, experts, score):
    g = torch.Generator(device="cuda").manual_seed(rows + experts)
    z = 3.0 * torch.randn(rows, experts, generator=g, device="cuda")
    b = 0.3 * torch.randn(experts, generator=g, device="cuda")
    for top in {1, min(8, experts), min(16, experts)}:
        for dt in (torch.float32, BF):
            for bias in (None, b):
                for ren, sc in ((True, 1.0), (False, 2.5)):
                    ids, w = fq.fp4_moe_route(z.to(dt), top, score=score, bias=bias, renormalize=ren, scale=sc)
                    i64, w64 = route64(z.to(dt), top, score, bias, ren, sc)
                    assert torch.equal(ids, i64)             # bf16 logits have ties
                    assert ((w.double() - w64).abs() <= 2.0 ** -23 * w64.abs()).all()


def test_route_masks_ties_and_nan():
    inf = float("inf")
    z = torch.tensor([[-inf, 1.0, -inf, 1.0, 0.5], [-inf] * 5, [0.0, 2.0, 2.0, 2.0, -0.0], [1.0, float("nan"), 5.0, -inf, 0.0],
                      [-200.0, -300.0, -inf, -250.0, -400.0]], device="cuda")
    ids, w = fq.fp4_moe_route(z, 3)
    assert ids.tolist()[:4] == [[1, 3, 4], [-1, -1, -1], [1, 2, 3], [1, 2, 0]]
    assert ids.tolist()[4] == [0, 3, 1]
    assert w[1].tolist() == [0.0] * 3 and torch.isnan(w[3]).all()
    assert torch.allclose(w[2], torch.full((3,), 1 / 3, device="cuda"), rtol=2.0 ** -23, atol=0)
    ids, w = fq.fp4_moe_route(z[:2], 4, score="sigmoid", bias=torch.tensor([9.0, 0, 9, 0, 1], device="cuda"))
    assert ids.tolist() == [[4, 1, 3, -1], [-1] * 4] and w[0, 3].item() == 0.0
    z = torch.full((2, 3), -2000.0, device="cuda")            # sigmoids of zero: no weight to share
    ids, w = fq.fp4_moe_route(z, 2, score="sigmoid")
    assert ids.tolist() == [[0, 1]] * 2 and w.tolist() == [[0.0, 0.0]] * 2


def test_route_strided_rows():
    z = torch.randn(9, 50, device="cuda")
    a, b = fq.fp4_moe_route(z[:, :41], 5), fq.fp4_moe_route(z[:, :41].contiguous(), 5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
