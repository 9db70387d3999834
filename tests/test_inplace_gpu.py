"""The in-place forms that the C ABI promises give the bits of the call whose
outputs lie elsewhere: the norms at a vector width, an odd one and one whose
backward takes two launches, and the adapters' wide-rank form."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _randn(g, *shape, sd=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * sd).to(dtype).cuda()


def _args(i, alpha, eps):
    x, r = i["x"], i["res"]
    return fq.Fp4NormC(x.data_ptr(), x.stride(0), r.data_ptr(), r.stride(0), x.shape[0], x.shape[1], i["w_pre"].data_ptr(),
                       i["w_post"].data_ptr(), i["gate"].data_ptr(), alpha, eps, fq.DTYPE[x.dtype], fq.DTYPE[r.dtype],
                       fq.DTYPE[i["w_pre"].dtype])


@pytest.mark.parametrize("rows,cols", [(300, 1024), (37, 1027), (5, 18944), (3, 32767)])
@pytest.mark.parametrize("xd,rd", [(BF, FP), (FP, BF), (BF, BF)])
def test_norms(rows, cols, xd, rd):
    g = torch.Generator().manual_seed(rows + cols)
    i = dict(x=_randn(g, rows, cols, dtype=xd), res=_randn(g, rows, cols, sd=2, dtype=rd),
             w_pre=_randn(g, cols, dtype=FP), w_post=_randn(g, cols, dtype=FP), gate=_randn(g, rows, dtype=FP))
    dn, dh = _randn(g, rows, cols, sd=0.1, dtype=xd), _randn(g, rows, cols, sd=0.1, dtype=rd)
    kw = dict(w_post=i["w_post"], gate=i["gate"], alpha=0.75)
    h, n, stats = fq.fp4_residual_norm(i["x"], i["res"], i["w_pre"], eps=1e-6, **kw)
    want = fq.fp4_residual_norm_backward(dn, dh, i["x"], i["res"], i["w_pre"], stats, **kw)
    L, stream = fq.lib(), torch.cuda.current_stream().cuda_stream
    # h on res, n on x
    j = dict(i, x=i["x"].clone(), res=i["res"].clone())
    st = torch.empty(rows, 2, device="cuda")
    assert L.fp4_residual_norm(ctypes.byref(_args(j, 0.75, 1e-6)), j["res"].data_ptr(), cols, j["x"].data_ptr(), cols,
                               st.data_ptr(), stream) == 0
    assert torch.equal(j["res"], h) and torch.equal(j["x"], n) and torch.equal(st, stats)
    need = L.fp4_residual_norm_workspace(rows, cols, 1)
    for dx_on, dres_on in (("x", "res"), ("dn", "dh"), ("x", "dh"), ("dn", "res")):
        j = dict(i, x=i["x"].clone(), res=i["res"].clone(), dn=dn.clone(), dh=dh.clone())
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        dw2, dw1, dg = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(rows, device="cuda")
        assert L.fp4_residual_norm_backward(ctypes.byref(_args(j, 0.75, 0.0)), stats.data_ptr(), j["dn"].data_ptr(), cols,
                                            j["dh"].data_ptr(), cols, j[dx_on].data_ptr(), cols, j[dres_on].data_ptr(), cols,
                                            dw2.data_ptr(), dw1.data_ptr(), dg.data_ptr(), ws.data_ptr(), need, stream) == 0
        got = (j[dx_on], j[dres_on], dw2, dw1, dg)
        for a, b, what in zip(got, (want.dx, want.dres, want.dw_pre, want.dw_post, want.dgate), ("dx", "dres", "w2", "w1", "g")):
            assert torch.equal(a, b), (dx_on, dres_on, what)


@pytest.mark.parametrize("m", [9, 100, 333])
@pytest.mark.parametrize("rank", [16, 64, 128])
def test_adapters(m, rank):
    """Several adapters and rows without one, in tiles of one adapter, of a few
    and of more than four."""
    g = torch.Generator().manual_seed(m + rank)
    n, k, la = 520, 264, 7
    x, dy, base, dxb = (_randn(g, m, c) for c in (k, n, n, k))
    bank = fq.LoraBank(_randn(g, la, rank, k, sd=0.1), _randn(g, la, n, rank, sd=0.1), _randn(g, la, dtype=FP))
    runs = torch.arange(m).mul(9).div(m, rounding_mode="floor") - 1
    for slots in (runs, torch.randint(-1, la, (m,), generator=g)):
        slots = slots.int().cuda()
        y, t = fq.fp4_lora_apply(x, bank, slots, base=base)
        here = base.clone()
        y2, t2 = fq.fp4_lora_apply(x, bank, slots, base=here, out=here)
        assert y2 is here and torch.equal(y, here) and torch.equal(t, t2)
        want = fq.fp4_lora_backward(dy, x, t, bank, slots, dx_base=dxb)
        here = dxb.clone()
        got = fq.fp4_lora_backward(dy, x, t, bank, slots, dx_base=here, dx=here)
        assert got[0] is here and all(torch.equal(a, b) for a, b in zip(want, got))
