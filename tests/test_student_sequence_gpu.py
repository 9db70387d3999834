"""The epilogue, mixture-of-experts and distillation calls together, as a
student with FP4 weights is trained from a teacher and served: every stage
against binary64 on that stage's own inputs (the tolerances of each call's
tests), calls on other streams, captured and replayed graphs, and rows past
32-bit offsets."""
import pytest
import torch

import fp4_block_scaled_quantize_amd as fq
from tests import test_distill_gpu as td
from tests import test_epilogue_gpu as te
from tests import test_moe_gpu as tm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _q(x, **kw):
    return fq.fp4_quantize(x, 16, "e4m3", **kw)


def test_training_step():
    """Two layers and the loss, forward and backward: products with their
    epilogues, the teacher's top list, the loss, and the gradients back through
    the products' transposes."""
    m, h, f, v, top = 96, 256, 512, 1000, 16
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s, sd=1.0):
        return (sd * torch.randn(*s, generator=g, device="cuda")).to(BF)
    x, wg, wu, wd, wv = r(m, h), r(f, h, sd=0.08), r(f, h, sd=0.08), r(h, f, sd=0.06), r(v, h, sd=0.1)
    bias = r(f, sd=0.1)
    qx, qg, qu, qd, qv = _q(x), _q(wg), _q(wu), _q(wd), _q(wv)
    up = fq.fp4_gemm(qx, qu)
    a, pre = fq.fp4_gemm_epilogue(qx, qg, bias=bias, act="silu", mul=up, save_pre=True)
    te.check(a, pre, *te.product64(qx, qg), "silu", bias, up, None)
    qa = _q(a)
    y, none = fq.fp4_gemm_epilogue(qa, qd, residual=x)
    assert none is None
    te.check(y, None, *te.product64(qa, qd), "none", None, None, x)
    qy = _q(y)
    z = fq.fp4_gemm(qy, qv)
    teacher = fq.fp4_token_logprobs((z.float() + 0.5 * torch.randn(m, v, generator=g, device="cuda")), top=top, temperature=2.0)
    gl = torch.full((m,), 1.0 / m, device="cuda")
    loss, dz = td.check(z, teacher.top_ids, teacher.top_logprobs, 2.0, g=gl)
    assert (loss.loss > 0).all()
    # back: dy = dz Wv, the residual's gradient is dy; da = dy Wd; the epilogue; dx = dpre Wg + dup Wu
    qdt, qgt, qut = (fq.fp4_quantize_transposed(w) for w in (wd, wg, wu))
    pad = torch.zeros(m, 24, dtype=BF, device="cuda")          # K of a product is a multiple of 128
    qvt = _q(torch.cat([wv, torch.zeros(24, h, dtype=BF, device="cuda")]).t().contiguous())
    dy = fq.fp4_gemm(_q(torch.cat([dz, pad], 1)), qvt)
    da = fq.fp4_gemm(_q(dy), qdt)
    d = fq.fp4_epilogue_backward(da, pre, act="silu", mul=up, bias=True)
    te.check_backward(d, da, pre, "silu", up, True)
    dup = fq.fp4_gemm(_q(d.dmul), qut)
    dx, _ = fq.fp4_gemm_epilogue(_q(d.dpre), qgt, mul=torch.ones_like(dy), residual=dup)
    te.check(dx, None, *te.product64(_q(d.dpre), qgt), "none", None, torch.ones_like(dy), dup)


def test_serving_step():
    """A decode batch: a dense block of weight-only products and a mixture-of-experts block on the same residual stream."""
    m, h, f, e, top = 5, 512, 768, 12, 3
    x = tm.tokens(m, h, 2)
    wg, wu, wd = (te.quantized(*s, 3 + i, 16, "e4m3", "e2m1", 0.05) for i, s in enumerate(((f, h), (f, h), (h, f))))
    up = fq.fp4_wo_gemm(x, wu)
    a = fq.fp4_wo_gemm_epilogue(x, wg, act="gelu_tanh", mul=up)
    te.check(a, None, *te.product64(x, wg), "gelu_tanh", None, up, None)
    y = fq.fp4_wo_gemm_epilogue(a, wd, residual=x)
    te.check(y, None, *te.product64(a, wd), "none", None, None, x)
    bank = tm.bank_of(e, h, f, 9)
    ids, w = fq.fp4_moe_route(y.float() @ torch.randn(h, e, device="cuda"), top, score="sigmoid", bias=torch.randn(e, device="cuda") * 0.1)
    out = fq.fp4_moe(y, bank, ids, w, residual=y)
    tm.check(out, y, bank, ids, w, residual=y)


def _everything():
    """(inputs, run): one of each call on shared inputs; run returns every output."""
    a, b = te.quantized(300, 4096, 30, 16, "e4m3", "e2m1", 1.0), te.quantized(520, 4096, 31, 16, "e4m3", "e2m1", 0.1)
    x, w = tm.tokens(4, 512, 32), te.quantized(264, 512, 33, 16, "e4m3", "e2m1", 0.1)
    bias, mul, res = te.tensors(300, 520, 34, BF, True, True)
    pre, dy, mu = (torch.randn(1500, 136, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).to(BF) for i in range(3))
    bank, t = tm.bank_of(9, 256, 384, 35), tm.tokens(7, 256, 36)
    logits = torch.randn(7, 9, device="cuda", generator=torch.Generator(device="cuda").manual_seed(37))
    z = td.student(6, 300000, 38, torch.float32)
    ids, lp = td.teacher(z, 12, 1.0, 0.4, 39)
    g = torch.rand(6, device="cuda") + 0.5
    assert fq.lib().fp4_gemm_epilogue_workspace(a.packed(), b.packed()) == 0
    live = [mul, res, x, pre, dy, mu, t, logits, z]

    def run(stream=None):
        was = fq.set_gemm_small_outputs(0)
        try:
            out = list(fq.fp4_gemm_epilogue(a, b, bias=bias, act="silu", mul=mul, residual=res, save_pre=True, stream=stream))
        finally:
            fq.set_gemm_small_outputs(was)
        out.append(fq.fp4_wo_gemm_epilogue(x, w, act="gelu", stream=stream))
        d = fq.fp4_epilogue_backward(dy, pre, act="silu", mul=mu, bias=True, stream=stream)
        out += [d.dpre, d.dbias, d.dmul]
        i, wt = fq.fp4_moe_route(logits, 3, stream=stream)
        out += [i, wt, fq.fp4_moe(t, bank, i, wt, stream=stream)]
        f = fq.fp4_distill_loss(z, ids, lp, stream=stream)
        return out + [f.loss, fq.fp4_distill_loss_backward(z, ids, lp, f, g, stream=stream)]
    return live, run


def test_streams():
    """On a stream given as an object, as a handle, and as the current one: the same bits, in that stream's order."""
    _, run = _everything()
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for how in (side, side.cuda_stream):
        got = run(stream=how)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.cuda.stream(side):
        got = run()
        zero = run(stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and all(torch.equal(p, q) for p, q in zip(zero, want))


def test_graphs_replay_with_new_inputs():
    """Captured twice, replayed in turn with new inputs and eager work between: each replay is the eager call."""
    live, run = _everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for rep in range(4):
        for t in live:
            t.copy_(torch.roll(t, rep + 1, 0))
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for graph, out in graphs[::1 if rep % 2 else -1]:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want)), rep


def test_offsets_past_32_bits():
    """Rows that start past 2^32 bytes: strided mul, residual, pre and outputs of a product, the epilogue's
    gradients, logits, and experts behind 4 GiB of others."""
    m, n, k = 3, 264, 256
    far = (1 << 31) + 1000                                     # elements: the last rows lie past 4 and 8 GiB
    a, b = te.quantized(m, k, 40, 16, "e4m3", "e2m1", 1.0), te.quantized(n, k, 41, 16, "e4m3", "e2m1", 0.1)
    v, e = te.product64(a, b)
    big = torch.empty(2 * far + n, dtype=BF, device="cuda")
    rows = big.as_strided((m, n), (far, 1))
    rows.copy_(torch.randn(m, n, device="cuda"))
    mul = rows.clone()
    for small in (0, 1 << 21):
        was = fq.set_gemm_small_outputs(small)
        try:
            te.check(fq.fp4_gemm_epilogue(a, b, act="silu", mul=rows, residual=rows)[0], None, v, e, "silu", None, mul, mul)
            keep = rows.clone()
            y, _ = fq.fp4_gemm_epilogue(a, b, residual=rows, out=rows)
            te.check(y.contiguous(), None, v, e, "none", None, None, keep)
            rows.copy_(keep)
        finally:
            fq.set_gemm_small_outputs(was)
    d = fq.fp4_epilogue_backward(rows, rows, act="silu", mul=rows, bias=True)
    te.check_backward(d, mul, mul, "silu", mul, True)
    z = td.student(m, n, 42, BF)
    rows.copy_(z)
    ids, lp = td.teacher(z, 5, 1.0, 0.3, 43)
    _, d = td.check(rows, ids, lp)
    f, g = fq.fp4_distill_loss(rows, ids, lp), torch.rand(m, device="cuda", generator=torch.Generator(device="cuda").manual_seed(m)) + 0.5
    fq.fp4_distill_loss_backward(rows, ids, lp, f, g, out=rows)
    assert torch.equal(rows, d)
    del big, rows
    # 80 experts of 192 and 96 MiB: the last ones' codes lie past 4 GiB on both sides
    e, h, ffn = 80, 4096, 24576

    def zeros(rows, cols):
        return fq.QTensor(torch.zeros(rows, cols, dtype=torch.uint8, device="cuda"),
                          torch.zeros(rows, cols // 32, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda"), rows, cols, 32,
                          "e8m0", amax="none", element="fp8_e4m3")
    up, down = zeros(e * 2 * ffn, h), zeros(e * h, ffn)
    last = tm.bank_of(1, h, ffn, 44, 32, "e8m0", "fp8_e4m3", each=False)
    for whole, one in ((up, last.gate_up), (down, last.down)):
        assert whole.q.numel() > 1 << 32
        whole.q[-one.rows:].copy_(one.q)
        whole.scales[-one.rows:].copy_(one.scales)
    x = tm.tokens(2, h, 45)
    ids = torch.tensor([[79, 0], [3, 79]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    zero = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    tm.check(fq.fp4_moe(x, fq.MoeBank(up, down, e), ids, w), x, last, zero, w[:, :1])     # the others are zeros
