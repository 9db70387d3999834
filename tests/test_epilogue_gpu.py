"""Products with bias, activation, multiplier and residual, and their
gradients, against binary64.

Tolerances.  The product's sums are within 1e-5 sum |a||w| (include/fp4.h) of
the exact ones; call that E.  An activation's slope is below 1.13, and its
binary32 value within (|v| + 8) 2^-22 of itself (an exponential whose argument
|v| log2 e was rounded once, and a few roundings).  Each further binary32 step
rounds by 2^-24, the output once by half a step, 2^-8 in bf16."""
import math

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
BF = torch.bfloat16


def act64(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.where(v != v, v, 0.0))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def tensors(m, n, seed, bias, mul, residual):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    return (None if bias is None else r(n).to(bias), r(m, n).to(BF) if mul else None,
            (3.0 * r(m, n)).to(BF) if residual else None)


def check(y, pre, v, e, act, bias, mul, residual):
    """y and pre against binary64 v (the product) with error bound e."""
    if bias is not None:
        v = v + bias.double()
    a = act64(v, act)
    scale = mul.double().abs() if mul is not None else 1.0
    want = a * mul.double() if mul is not None else a
    tol = scale * (1.13 * (e + 2.0 ** -23 * v.abs()) + (v.abs() + 8.0) * 2.0 ** -22 * a.abs())
    if residual is not None:
        want = want + residual.double()
    tol = tol + 2.0 ** -22 * want.abs() + 2.0 ** -8 * want.abs() + 1e-37
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), (y.double() - want).abs().max().item())
    if pre is not None:
        bad = (pre.double() - v).abs() > e + 2.0 ** -22 * v.abs() + 2.0 ** -8 * v.abs()
        assert not bad.any(), int(bad.sum())


def quantized(m, k, seed, block, scale, element, sd):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, k, generator=g, device="cuda") * sd
    amax = "none" if scale == "e8m0" else "current"
    return fq.fp4_quantize(x.to(BF), block, scale, amax=amax, element=element)


def product64(a, b):
    x = a.double() if isinstance(a, torch.Tensor) else fq.fp4_dequantize(a).double()
    w = fq.fp4_dequantize(b).double()
    return x @ w.t(), 1e-5 * (x.abs() @ w.abs().t())


# every kernel of the products: (block, scale, element, K), with the bound on
# small products (0: the tiled kernels)
PATHS = [(32, "e8m0", "e2m1", 512, 0), (32, "e8m0", "e2m1", 384, 0), (16, "e8m0", "e2m1", 512, 0),
         (16, "e8m0", "e2m1", 128, 0), (16, "e4m3", "e2m1", 256, 0), (32, "e4m3", "e2m1", 128, 0),
         (16, "e3m4", "e2m1", 256, 0), (16, "ue5m3", "e2m1", 256, 0), (32, "e8m0", "fp8_e4m3", 256, 0),
         (16, "e4m3", "int8", 256, 0), (32, "e8m0", "int4", 256, 0), (16, "e4m3", "int4", 128, 0),
         (32, "e8m0", "fp6_e2m3", 256, 0), (32, "e8m0", "fp6_e3m2", 256, 0), (32, "e8m0", "int6", 256, 0),
         (32, "e8m0", "int8", 256, 0),
         (16, "e4m3", "e2m1", 256, 1 << 21), (16, "e3m4", "e2m1", 256, 1 << 21), (32, "e8m0", "e2m1", 256, 1 << 21),
         (16, "ue5m3", "e2m1", 256, 1 << 21), (16, "e8m0", "e2m1", 256, 1 << 21), (32, "e8m0", "fp8_e4m3", 256, 1 << 21),
         (16, "e4m3", "int8", 256, 1 << 21)]


@pytest.mark.parametrize("block,scale,element,k,small", PATHS)
def test_product_epilogue_on_every_path(block, scale, element, k, small):
    m, n = 157, 333                                        # neither a multiple of a tile, nor rows of whole vectors
    a = quantized(m, k, 1, block, scale, element, 1.0)
    b = quantized(n, k, 2, block, scale, element, 0.1)
    v, e = product64(a, b)
    was = fq.set_gemm_small_outputs(small)
    try:
        for i, act in enumerate(ACTS):
            bias, mul, res = tensors(m, n, 10 + i, [None, torch.float32, BF][i % 3], i % 2 == 0, i % 3 != 1)
            y, pre = fq.fp4_gemm_epilogue(a, b, bias=bias, act=act, mul=mul, residual=res, save_pre=i != 3)
            check(y, pre, v, e, act, bias, mul, res)
    finally:
        fq.set_gemm_small_outputs(was)


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 256, 256), (256, 256, 128), (257, 264, 640), (700, 512, 1024), (33, 8, 256)])
@pytest.mark.parametrize("scale,block", [("e8m0", 32), ("e4m3", 16)])
def test_product_epilogue_sizes(m, n, k, scale, block):
    a = quantized(m, k, 3, block, scale, "e2m1", 1.0)
    b = quantized(n, k, 4, block, scale, "e2m1", 0.1)
    v, e = product64(a, b)
    for small in (0, 1 << 21):
        was = fq.set_gemm_small_outputs(small)
        try:
            bias, mul, res = tensors(m, n, 5, BF, True, True)
            y, pre = fq.fp4_gemm_epilogue(a, b, bias=bias, act="silu", mul=mul, residual=res, save_pre=True)
            check(y, pre, v, e, "silu", bias, mul, res)
        finally:
            fq.set_gemm_small_outputs(was)


@pytest.mark.parametrize("block,scale,element,k", [(32, "e8m0", "e2m1", 2304), (32, "e8m0", "e2m1", 4096), (32, "e8m0", "e2m1", 2176),
                                                   *((b, s, e, 1408 if b == 32 or s != "e8m0" else 2304)
                                                     for b, s, e, _, small in PATHS if not small and (b, s, e) != (32, "e8m0", "e2m1"))])
def test_product_epilogue_in_k_ranges(block, scale, element, k):
    """Few tiles of a long K: ranges of it, the last one short, joined before the epilogue."""
    m, n = 260, 301
    a, b = quantized(m, k, 61, block, scale, element, 1.0), quantized(n, k, 62, block, scale, element, 0.1)
    v, e = product64(a, b)
    was = fq.set_gemm_small_outputs(0)
    try:
        assert fq.lib().fp4_gemm_epilogue_workspace(a.packed(), b.packed()) >= 2 * 4 * m * 304
        bias, mul, res = tensors(m, n, 63, BF, True, True)
        y, pre = fq.fp4_gemm_epilogue(a, b, bias=bias, act="silu", mul=mul, residual=res, save_pre=True)
        check(y, pre, v, e, "silu", bias, mul, res)
        for _ in range(3):
            assert torch.equal(fq.fp4_gemm_epilogue(a, b, bias=bias, act="silu", mul=mul, residual=res)[0], y)
    finally:
        fq.set_gemm_small_outputs(was)


@pytest.mark.parametrize("small", [0, 1 << 21])
def test_product_epilogue_strided_rows_stay_inside(small):
    """Padded rows of every operand, and y in the place of the residual; what lies behind the rows stays."""
    m, n, k = 130, 300, 256
    a = quantized(m, k, 6, 16, "e4m3", "e2m1", 1.0)
    b = quantized(n, k, 7, 16, "e4m3", "e2m1", 0.1)
    v, e = product64(a, b)
    was = fq.set_gemm_small_outputs(small)
    try:
        for pad in (4, 1):                                 # rows of whole vectors, and none
            _, mul, res = tensors(m, n + pad, 8, None, True, True)
            keep, want = res.clone(), res[:, :n].clone()
            y, _ = fq.fp4_gemm_epilogue(a, b, act="gelu", mul=mul[:, :n], residual=res[:, :n], out=res[:, :n])
            assert y.data_ptr() == res.data_ptr()
            check(y, None, v, e, "gelu", None, mul[:, :n], want)
            assert torch.equal(res[:, n:], keep[:, n:])
    finally:
        fq.set_gemm_small_outputs(was)


@pytest.mark.parametrize("m", [1, 2, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("n,k", [(512, 256), (8200, 512), (33, 1024)])
def test_weight_only_epilogue(m, n, k):
    w = quantized(n, k, 20 + m, 16, "e4m3", "e2m1", 0.1)
    x = torch.randn(m, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(m)).to(BF)
    v, e = product64(x, w)
    for i, act in enumerate(ACTS):
        bias, mul, res = tensors(m, n, 30 + i, [torch.float32, BF, None][i % 3], i % 2 == 1, i != 1)
        check(fq.fp4_wo_gemm_epilogue(x, w, bias=bias, act=act, mul=mul, residual=res), None, v, e, act, bias, mul, res)


@pytest.mark.parametrize("block,scale,element", [(32, "e8m0", "e2m1"), (16, "e1m6", "e2m1"), (32, "e8m0", "int4"), (32, "e8m0", "fp8_e4m3"),
                                                 (16, "e4m3", "int8"), (32, "e8m0", "fp6_e2m3"), (32, "e8m0", "fp6_e3m2"),
                                                 (16, "e4m3", "int6")])
def test_weight_only_epilogue_grids(block, scale, element):
    m, n, k = 7, 160, 512
    w = quantized(n, k, 40, block, scale, element, 0.1)
    x = torch.randn(m, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(41)).to(BF)
    v, e = product64(x, w)
    bias, mul, res = tensors(m, n, 42, BF, True, True)
    check(fq.fp4_wo_gemm_epilogue(x, w, bias=bias, act="gelu_tanh", mul=mul, residual=res), None, v, e, "gelu_tanh", bias,
          mul, res)


def test_plain_epilogue_has_the_products_bits():
    """Without any part the epilogue is the product itself, on both products."""
    a, b = quantized(100, 256, 50, 16, "e4m3", "e2m1", 1.0), quantized(333, 256, 51, 16, "e4m3", "e2m1", 0.1)
    assert torch.equal(fq.fp4_gemm_epilogue(a, b)[0], fq.fp4_gemm(a, b))
    x = torch.randn(5, 256, device="cuda").to(BF)
    assert torch.equal(fq.fp4_wo_gemm_epilogue(x, b), fq.fp4_wo_gemm(x, b))


def test_extreme_values_of_the_activations():
    """Far values, infinities and NaN through the epilogue: the weight is one, so v is the bias."""
    vals = [0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, -12.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38,
            float("inf"), float("nan")]
    n = len(vals)
    x = torch.zeros(1, 256, device="cuda", dtype=BF)
    w = quantized(n, 256, 52, 16, "e4m3", "e2m1", 0.1)
    b = torch.tensor(vals, device="cuda")
    for act in ACTS:
        y = fq.fp4_wo_gemm_epilogue(x, w, bias=b, act=act)[0].double()
        want = act64(b.double(), act)
        for i, v in enumerate(vals):
            if v != v:
                assert math.isnan(y[i].item())
            elif math.isinf(v) or abs(want[i].item()) > 3e38:
                assert y[i].item() == math.inf or abs(y[i].item()) > 3e38
            else:
                # a value below binary32's normal range may be flushed
                assert abs(y[i].item() - want[i].item()) <= (2.0 ** -8 + (abs(v) + 8.0) * 2.0 ** -22) * abs(want[i].item()) + 1e-37, (act, v)


# ---------------------------------------------------------------------------
def slope64(v, act):
    v = v.clone().requires_grad_(True)
    return torch.autograd.grad(act64(v, act).sum(), v)[0]


def check_backward(d, dy, pre, act, mul, bias):
    """Slopes are within (|v| + 16) 2^-21 of 1 + |slope|: the same exponential, and products of a few of its kind."""
    v, g = pre.double(), dy.double()
    s = torch.where(v > 0, 1.0, 0.0).double() if act == "relu" else slope64(v, act) if act != "none" else torch.ones_like(v)
    u = g * mul.double() if mul is not None else g
    want = u * s
    err = u.abs() * (v.abs() + 16.0) * 2.0 ** -21 * (1.0 + s.abs())
    if act == "none":
        err = want.abs() * 2.0 ** -23
    assert ((d.dpre.double() - want).abs() <= err + 2.0 ** -8 * want.abs() + 1e-37).all()
    if mul is not None:
        a = act64(v, act)
        w = g * a
        assert ((d.dmul.double() - w).abs() <= w.abs() * ((v.abs() + 8.0) * 2.0 ** -22 + 2.0 ** -8) + 1e-37).all()
    else:
        assert d.dmul is None
    if bias:
        # a sum of at most rows terms in binary32: rows 2^-24 of their sizes, far above the order that is used
        w = want.sum(0)
        assert ((d.dbias.double() - w).abs() <= err.sum(0) + want.shape[0] * 2.0 ** -24 * want.abs().sum(0) + 1e-37).all()
    else:
        assert d.dbias is None


@pytest.mark.parametrize("m,n", [(1, 1), (1, 264), (3, 7), (31, 256), (130, 1027), (513, 300), (2000, 64), (0, 40)])
@pytest.mark.parametrize("act", ACTS)
def test_backward(m, n, act):
    g = torch.Generator(device="cuda").manual_seed(m * 7 + n)
    pre = (2.0 * torch.randn(m, n, generator=g, device="cuda")).to(BF)
    dy = torch.randn(m, n, generator=g, device="cuda").to(BF)
    mul = torch.randn(m, n, generator=g, device="cuda").to(BF)
    for mu in (None, mul):
        for bias in (False, True):
            d = fq.fp4_epilogue_backward(dy, pre, act=act, mul=mu, bias=bias)
            check_backward(d, dy, pre, act, mu, bias)


@pytest.mark.parametrize("m,n", [(1024, 513), (1025, 513), (1056, 1031), (45000, 8), (33000, 519), (1200, 11008)])
def test_backward_of_many_row_ranges(m, n):
    """Either side of the rows that one launch sums, one range to a thousand."""
    test_backward(m, n, "gelu_tanh")


def test_backward_strided_rows():
    m, n = 70, 200
    t = [torch.randn(m, n + p, device="cuda").to(BF)[:, :n] for p in (8, 3, 16)]
    d = fq.fp4_epilogue_backward(t[0], t[1], act="silu", mul=t[2], bias=True)
    check_backward(d, t[0], t[1], "silu", t[2], True)


def test_backward_without_activation_needs_no_pre():
    dy = torch.randn(90, 33, device="cuda").to(BF)
    d = fq.fp4_epilogue_backward(dy, None, bias=True)
    assert d.dpre is dy
    assert ((d.dbias.double() - dy.double().sum(0)).abs() <= 90 * 2.0 ** -24 * dy.double().abs().sum(0)).all()
    d = fq.fp4_epilogue_backward(dy, None)
    assert d.dpre is dy and d.dbias is None


def test_backward_far_values():
    """Slopes at far values are 0 or 1, never NaN."""
    v = torch.tensor([[-3e38, -1e20, -1e4, -200.0, -90.0, 90.0, 200.0, 1e4, 1e20, 3e38]], device="cuda").to(BF)
    dy = torch.ones_like(v)
    for act in ACTS[1:]:
        d = fq.fp4_epilogue_backward(dy, v, act=act).dpre.double()
        assert torch.equal(d[0, 5:], torch.ones(5, device="cuda").double()) and (d[0, :5].abs() <= 1e-30).all(), act


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """The backward call's slope against central differences of the forward
    formula in binary64, step 2^-10: the third derivatives are below 3, so they
    are 3 / 6 2^-20 off, and relu is kept off its corner."""
    v = torch.linspace(-6.0, 6.0, 1001, device="cuda").to(BF)[None]
    v = v[:, v[0].abs() > 2.0 ** -8].contiguous()
    h = 2.0 ** -10
    want = (act64(v.double() + h, act) - act64(v.double() - h, act)) / (2 * h)
    d = fq.fp4_epilogue_backward(torch.ones_like(v), v, act=act).dpre.double()
    assert ((d - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16).all()


@pytest.mark.parametrize("m,n", [(70, 203), (1500, 519)])    # one launch, and ranges of rows
@pytest.mark.parametrize("to", [("dy", "pre"), ("pre", "mul"), ("mul", "dy"), ("dy", "mul")])
def test_backward_in_place(m, n, to):
    """dpre and dmul in the place of two of the inputs, padded rows: the bits of the call into rows of their own."""
    g = torch.Generator(device="cuda").manual_seed(m + n)
    t = {k: torch.randn(m, n + 5, generator=g, device="cuda").to(BF) for k in ("dy", "pre", "mul")}
    behind = {k: v[:, n:].clone() for k, v in t.items()}
    want = fq.fp4_epilogue_backward(t["dy"][:, :n], t["pre"][:, :n], act="gelu_tanh", mul=t["mul"][:, :n], bias=True)
    lib, ld, dbias = fq.lib(), n + 5, torch.empty(n, device="cuda")
    ws = torch.empty(max(16, lib.fp4_epilogue_workspace(m, n)), dtype=torch.uint8, device="cuda")
    args = [x for k in ("dy", "pre", "mul") for x in (t[k].data_ptr(), ld)]
    st = lib.fp4_epilogue_backward(*args, m, n, fq.ACT["gelu_tanh"], t[to[0]].data_ptr(), ld, t[to[1]].data_ptr(), ld,
                                   dbias.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(t[to[0]][:, :n], want.dpre) and torch.equal(t[to[1]][:, :n], want.dmul) and torch.equal(dbias, want.dbias)
    assert all(torch.equal(t[k][:, n:], behind[k]) for k in t)


@pytest.mark.parametrize("place", ["mul", "residual"])
@pytest.mark.parametrize("block,scale,k", [(32, "e8m0", 4096), (16, "e4m3", 1408)])
def test_product_epilogue_in_k_ranges_in_place(block, scale, k, place):
    m, n = 260, 301
    a, b = quantized(m, k, 71, block, scale, "e2m1", 1.0), quantized(n, k, 72, block, scale, "e2m1", 0.1)
    bias, mul, res = tensors(m, n + 3, 73, torch.float32, True, True)
    bias, mul, res = bias[:n], mul[:, :n], res[:, :n]
    was = fq.set_gemm_small_outputs(0)
    try:
        assert fq.lib().fp4_gemm_epilogue_workspace(a.packed(), b.packed()) > 0
        want, pre = fq.fp4_gemm_epilogue(a, b, bias=bias, act="gelu", mul=mul, residual=res, save_pre=True)
        to = mul if place == "mul" else res
        y, p = fq.fp4_gemm_epilogue(a, b, bias=bias, act="gelu", mul=mul, residual=res, save_pre=True, out=to)
        assert y.data_ptr() == to.data_ptr() and torch.equal(y, want) and torch.equal(p, pre)
    finally:
        fq.set_gemm_small_outputs(was)


def test_gelu_slope_in_binary32():
    """At every bf16 number up to 13, as the sum of a single row, which nothing rounds to bf16: Phi(v) + v phi(v) with
    the normal tail within 2^-21 and exp(-v^2 / 2) within 2^-22 of itself, three roundings on the way to v phi(v) (a
    constant and two products), one of 1 - tail and one of the sum."""
    bits = torch.arange(0x2000, 0x4151, dtype=torch.int32)   # 2^-63 .. 13
    v = torch.cat([bits, bits + 0x8000 - 0x10000]).to(torch.int16).view(BF).cuda()[None]
    d = fq.fp4_epilogue_backward(torch.ones_like(v), v, act="gelu", bias=True).dbias.double().cpu()
    x = v[0].double().cpu()
    assert x.max() == 13.0 and x.min() == -13.0
    tail = 0.5 * torch.special.erfc(x.abs() / math.sqrt(2.0))
    vphi = x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    want = torch.where(x < 0, tail, 1.0 - tail) + vphi
    tol = 2.0 ** -21 * tail + (2.0 ** -22 + 3 * 2.0 ** -24) * vphi.abs() + 2.0 ** -24 * (want.abs() + (x >= 0))
    assert ((d - want).abs() <= tol).all(), ((d - want).abs() / tol).max()


def test_backward_bits_repeat():
    m, n = 3000, 500
    pre, dy, mul = ((torch.randn(m, n, device="cuda")).to(BF) for _ in range(3))
    a = fq.fp4_epilogue_backward(dy, pre, act="silu", mul=mul, bias=True)
    for _ in range(3):
        b = fq.fp4_epilogue_backward(dy, pre, act="silu", mul=mul, bias=True)
        assert torch.equal(a.dbias, b.dbias) and torch.equal(a.dpre, b.dpre) and torch.equal(a.dmul, b.dmul)
