"""Host-side checks of the epilogue, mixture-of-experts and distillation calls
that need no GPU: invalid arguments are refused before any launch (the
pointers are never dereferenced), workspaces have the sizes the calls ask
for, and the binding refuses what does not fit the kernels."""
import ctypes

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq

FAKE = 0x10000      # 16-byte aligned, never dereferenced: validation fails first
ROOM = 1 << 40
MANY = 1 << 39      # a row stride whose products no tensor has


def _q(rows, cols, block=16, scale=0, element=0, transform=0, q=FAKE, s=FAKE):
    return fq.Fp4TensorC(q, s, FAKE, rows, cols, fq.Fp4Format(block, scale, 0, 1, transform, 5 if transform else 0, element))


def _epi(bias=FAKE, bd=0, act=2, mul=FAKE, ldm=64, res=FAKE, ldr=64, pre=None, ldp=64):
    return fq.Fp4EpilogueC(bias, bd, act, mul, ldm, res, ldr, pre, ldp)


EPI = [(dict(act=-1), -1), (dict(act=5), -1), (dict(bd=2), -1), (dict(bias=FAKE + 2), -4), (dict(bias=FAKE + 1, bd=1), -4),
       (dict(ldm=63), -3), (dict(ldr=63), -3), (dict(mul=FAKE + 1), -4), (dict(res=FAKE + 1), -4), (dict(ldm=MANY), -2),
       (dict(mul=FAKE + 1024, ldm=72), -3), (dict(res=FAKE + 1024, ldr=72), -3)]
Y = FAKE + 1024


@pytest.mark.parametrize("kw,want", EPI + [(dict(pre=FAKE + 1), -4), (dict(pre=FAKE + 2, ldp=63), -3), (dict(pre=Y), -1),
                                           (dict(pre=FAKE), -1)])
def test_gemm_epilogue_rejects_before_launch(kw, want):
    a, b, e = _q(5, 256), _q(64, 256), _epi(**kw)
    assert fq.lib().fp4_gemm_epilogue(ctypes.byref(a), ctypes.byref(b), ctypes.byref(e), Y, 64, FAKE, ROOM, None) == want


@pytest.mark.parametrize("kw,want", EPI + [(dict(pre=FAKE + 512), -2)])
def test_wo_gemm_epilogue_rejects_before_launch(kw, want):
    w, e = _q(64, 256), _epi(**kw)
    assert fq.lib().fp4_wo_gemm_epilogue(FAKE, 256, 4, ctypes.byref(w), ctypes.byref(e), Y, 64, None) == want


def test_products_epilogues_refuse_what_the_products_refuse():
    L, e = fq.lib(), _epi()

    def gemm(a, b, y=Y, ldy=64, e=e, ws=FAKE, room=ROOM):
        return L.fp4_gemm_epilogue(ctypes.byref(a), ctypes.byref(b), None if e is None else ctypes.byref(e), y, ldy, ws, room, None)

    def wo(w, m=4, x=FAKE, ldx=256, y=Y, ldy=64, e=e):
        return L.fp4_wo_gemm_epilogue(x, ldx, m, ctypes.byref(w), None if e is None else ctypes.byref(e), y, ldy, None)
    ok = _q(64, 256)
    assert gemm(_q(5, 256), ok, e=None) == -1 and wo(ok, e=None) == -1
    assert gemm(_q(5, 256), ok, y=None) == -1 and gemm(_q(5, 256), ok, ldy=63) == -3 and gemm(_q(5, 256), ok, y=Y + 1) == -4
    assert gemm(_q(5, 128), ok) == -3 and gemm(_q(5, 0), _q(64, 0)) == -3 and gemm(_q(5, 256, 32, 4), ok) == -2
    assert gemm(_q(5, 256, q=FAKE + 4), ok) == -4 and gemm(_q(5, 256, transform=1), ok) == -2
    assert gemm(_q(5, 256, 16, 4, 3), _q(64, 256, 16, 2, 3)) == -2                 # a pairing without an exact type
    a, b = _q(3000, 4096), _q(800, 4096)                  # K in ranges
    need = L.fp4_gemm_epilogue_workspace(ctypes.byref(a), ctypes.byref(b))
    e2 = _epi(mul=None, res=None)
    assert need > 0 and need % (4 * 3000 * 800) == 0
    assert gemm(a, b, ldy=800, e=e2, ws=None) == -1 and gemm(a, b, ldy=800, e=e2, room=need - 1) == -1
    assert gemm(a, b, ldy=800, e=e2, ws=FAKE + 8) == -4
    assert L.fp4_gemm_epilogue_workspace(ctypes.byref(_q(5, 256)), ctypes.byref(ok)) == 0
    assert L.fp4_gemm_epilogue_workspace(None, ctypes.byref(ok)) == -1 and L.fp4_gemm_epilogue_workspace(ctypes.byref(ok), None) == -1
    assert wo(ok, m=0) == -2 and wo(ok, m=17) == -2 and wo(ok, x=None) == -1 and wo(ok, ldx=260) == -4
    # x as the output, be it the residual or not
    square = _q(256, 256)
    assert wo(square, y=FAKE, ldy=256, e=_epi(mul=None, res=None)) == -1
    assert wo(square, y=FAKE, ldy=256, e=_epi(mul=None, res=FAKE, ldr=256)) == -1
    assert wo(_q(64, 0)) == -3 and wo(_q(0, 256), ldy=0) == -3 and wo(_q(64, 256, transform=1)) == -2


def _back(dy=FAKE, ldy=64, pre=FAKE + 256, ldp=64, mul=FAKE + 512, ldm=64, rows=40, cols=64, act=2, dpre=FAKE + 1024, ldd=64,
          dmul=FAKE + 2048, ldg=64, db=FAKE, ws=FAKE, room=ROOM):
    return fq.lib().fp4_epilogue_backward(dy, ldy, pre, ldp, mul, ldm, rows, cols, act, dpre, ldd, dmul, ldg, db, ws, room, None)


@pytest.mark.parametrize("kw,want", [
    (dict(act=7), -1), (dict(rows=-1), -3), (dict(cols=0), -3), (dict(cols=(1 << 24) + 8, ldy=1 << 25), -2), (dict(rows=1 << 40), -2),
    (dict(dy=None), -1), (dict(pre=None), -1), (dict(dpre=None), -1), (dict(dmul=None), -1), (dict(dpre=FAKE + 2048), -1),
    (dict(ldy=63), -3), (dict(ldp=63), -3), (dict(ldm=63), -3), (dict(ldd=63), -3), (dict(ldg=63), -3), (dict(ldy=MANY), -2),
    (dict(dy=FAKE + 1), -4), (dict(pre=FAKE + 1), -4), (dict(mul=FAKE + 1), -4), (dict(dpre=FAKE + 1), -4), (dict(dmul=FAKE + 1), -4),
    (dict(dpre=FAKE, ldd=72), -3), (dict(dpre=FAKE + 256, ldd=72), -3), (dict(dmul=FAKE + 512, ldg=72), -3), (dict(dmul=FAKE, ldg=72), -3),
    (dict(db=FAKE + 2), -4), (dict(rows=2000, ws=None), -1), (dict(rows=2000, room=255), -1), (dict(rows=2000, ws=FAKE + 8), -4),
    (dict(rows=2000, mul=None, act=0, dpre=None, ws=None), -1),
])
def test_epilogue_backward_rejects_before_launch(kw, want):
    assert _back(**kw) == want


def test_epilogue_backward_with_nothing_to_do():
    assert _back(act=0, mul=None, pre=None, dpre=None, dmul=None, db=None, ws=None, room=0) == 0
    assert _back(rows=0, dy=None, pre=None, mul=None, dpre=None, dmul=None, db=None) == 0
    need = fq.lib().fp4_epilogue_workspace
    assert need(-1, 8) == -3 and need(8, 0) == -3 and need(1, (1 << 24) + 1) == -2
    for m in (0, 1, 31, 1000, 100000):
        for n in (1, 255, 257, 11008):
            # few rows are summed by one launch
            assert need(m, n) == 0 if m <= 1024 else 4 * n <= need(m, n) <= 4 * n * min(2048, (m + 31) // 32) + 16


def _moe(m=4, top=2, hidden=256, ffn=128, experts=3, x=FAKE, ldx=256, up=None, down=None, us=FAKE, ds=FAKE, ids=FAKE, w=FAKE, act=2,
         res=None, ldr=256, y=Y, ldy=256, ws=FAKE, room=ROOM, bank=True):
    up = up or _q(experts * 2 * ffn, hidden)
    down = down or _q(experts * hidden, ffn)
    b = fq.Fp4MoeBankC(up, down, us, ds, experts)
    return fq.lib().fp4_moe(x, ldx, m, ctypes.byref(b) if bank else None, ids, w, top, act, res, ldr, y, ldy, ws, room, None)


@pytest.mark.parametrize("kw,want", [
    (dict(bank=False), -1), (dict(act=9), -1), (dict(x=None), -1), (dict(y=None), -1), (dict(ids=None), -1), (dict(w=None), -1),
    (dict(m=0), -2), (dict(m=17), -2), (dict(top=0), -3), (dict(top=17), -2), (dict(experts=65536), -2),
    (dict(up=_q(767, 256)), -3), (dict(down=_q(769, 128)), -3), (dict(hidden=192, ldx=256), -3), (dict(ffn=64), -3),
    (dict(up=_q(768, 256, transform=1)), -2), (dict(up=_q(768, 256, q=FAKE + 8)), -4), (dict(down=_q(768, 128, s=FAKE + 2)), -4),
    (dict(down=_q(768, 128, 8)), -1), (dict(us=FAKE + 2), -4), (dict(ds=FAKE + 1), -4),
    (dict(ldx=255), -3), (dict(ldy=255), -3), (dict(res=FAKE, ldr=255), -3), (dict(ldx=1 << 40), -2), (dict(res=Y, ldr=264), -3),
    (dict(x=FAKE + 8), -4), (dict(ldx=260), -4), (dict(y=Y + 1), -4), (dict(res=FAKE + 1), -4), (dict(ids=FAKE + 2), -4),
    (dict(w=FAKE + 2), -4), (dict(ws=None), -1), (dict(room=4095), -1), (dict(ws=FAKE + 8), -4),
])
def test_moe_rejects_before_launch(kw, want):
    assert _moe(**kw) == want


def test_moe_refuses_an_expert_of_4_gib():
    # 2^32 bytes of one expert's gate and up codes
    assert _moe(ffn=1 << 18, hidden=1 << 14, ldx=1 << 14, ldy=1 << 14, experts=1, up=_q(1 << 19, 1 << 14), down=_q(1 << 14, 1 << 18)) == -2


def test_moe_workspace():
    need = fq.lib().fp4_moe_workspace
    assert need(-1, 2, 128) == -3 and need(1, 0, 128) == -3 and need(1, 1, 0) == -3 and need(17, 1, 8) == -2 and need(1, 17, 8) == -2
    assert need(4, 2, 128) == 4 * 4 * 2 * 128 and need(0, 2, 128) == 0


def _route(z=FAKE, dt=0, ld=8, rows=4, experts=8, top=2, score=0, bias=None, ren=1, scale=1.0, ids=FAKE, w=FAKE):
    return fq.lib().fp4_moe_route(z, dt, ld, rows, experts, top, score, bias, ren, scale, ids, w, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), -1), (dict(score=2), -1), (dict(scale=float("nan")), -1), (dict(rows=-1), -3), (dict(experts=0), -3), (dict(ld=7), -3),
    (dict(top=0), -3), (dict(top=9), -3), (dict(rows=1 << 22), -2), (dict(experts=1025, ld=1025), -2), (dict(experts=64, ld=64, top=17), -2),
    (dict(z=None), -1), (dict(ids=None), -1), (dict(w=None), -1), (dict(z=FAKE + 2), -4), (dict(bias=FAKE + 2), -4), (dict(ids=FAKE + 2), -4),
    (dict(w=FAKE + 1), -4), (dict(ld=MANY), -2),
])
def test_route_rejects_before_launch(kw, want):
    assert _route(**kw) == want
    assert _route(rows=0, z=None, ids=None, w=None) == 0


def _distill(z=FAKE, dt=1, ld=1000, n=4, v=1000, ids=FAKE, lp=FAKE, top=5, temp=1.0, rest=0, loss=FAKE, st=FAKE, ws=FAKE, room=ROOM):
    return fq.lib().fp4_distill_loss(z, dt, ld, n, v, ids, lp, top, temp, rest, loss, st, ws, room, None)


DISTILL = [(dict(dt=2), -1), (dict(temp=0.0), -1), (dict(temp=float("inf")), -1), (dict(temp=4e-39), -1), (dict(rest=2), -1), (dict(n=-1), -3),
           (dict(v=0), -3), (dict(ld=999), -3), (dict(top=0), -3), (dict(top=129), -2), (dict(v=(1 << 24) + 1, ld=1 << 25), -2),
           (dict(n=1 << 22), -2), (dict(z=None), -1), (dict(z=FAKE + 1), -4), (dict(ids=None), -1), (dict(lp=None), -1),
           (dict(ids=FAKE + 2), -4), (dict(lp=FAKE + 2), -4)]


@pytest.mark.parametrize("kw,want", DISTILL + [(dict(loss=None), -1), (dict(st=None), -1), (dict(loss=FAKE + 2), -4), (dict(st=FAKE + 2), -4),
                                               (dict(v=1 << 20, ld=1 << 20, ws=None), -1), (dict(v=1 << 20, ld=1 << 20, room=8), -1),
                                               (dict(v=1 << 20, ld=1 << 20, ws=FAKE + 4), -4)])
def test_distill_rejects_before_launch(kw, want):
    assert _distill(**kw) == want


@pytest.mark.parametrize("kw,want", DISTILL + [(dict(st=None), -1), (dict(g=None), -1), (dict(d=None), -1), (dict(ldd=999), -3),
                                               (dict(d=FAKE, ldd=1008), -3), (dict(ldd=MANY), -2), (dict(d=FAKE + 1), -4),
                                               (dict(st=FAKE + 2), -4), (dict(g=FAKE + 2), -4)])
def test_distill_backward_rejects_before_launch(kw, want):
    a = dict(z=FAKE, dt=1, ld=1000, n=4, v=1000, ids=FAKE, lp=FAKE, top=5, temp=1.0, rest=0, st=FAKE, g=FAKE, d=FAKE + 64, ldd=None)
    a.update(kw)
    if a["ldd"] is None:
        a["ldd"] = max(a["ld"], a["v"], 1)
    assert fq.lib().fp4_distill_loss_backward(*a.values(), None) == want


def test_distill_workspace():
    need = fq.lib().fp4_distill_workspace
    assert need(-1, 5, 0) == -3 and need(1, 0, 0) == -3 and need(1, (1 << 24) + 1, 0) == -2 and need(1 << 22, 8, 1) == -2 and need(1, 8, 2) == -1
    # rows of 512 KiB are whole, longer ones are cut unless there are many
    assert need(0, 128000, 0) == 0 and need(1, 131072, 0) == 0 and need(1, 262144, 1) == 0 and need(512, 200000, 0) == 0
    assert 0 < need(1, 131073, 0) <= 8 * 64 and 0 < need(1, 262145, 1) <= 8 * 64 and need(1000, 1 << 24, 1) == 8 * 1000 * 64


class _NoCalls:
    """Stands in for the library: any call is a test failure."""
    def __getattr__(self, name):
        raise AssertionError(f"library function {name} reached")


def test_binding_checks_before_any_call(monkeypatch):
    monkeypatch.setattr(fq, "lib", lambda: _NoCalls())
    bf = torch.bfloat16
    a, w = fq.QTensor.empty(4, 256, 16, "e4m3", device="cpu"), fq.QTensor.empty(64, 256, 16, "e4m3", device="cpu")
    x, y, b = torch.zeros(4, 256, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(64)
    up, down = fq.QTensor.empty(2 * 2 * 128, 256, 16, "e4m3", device="cpu"), fq.QTensor.empty(2 * 256, 128, 16, "e4m3", device="cpu")
    bank = fq.MoeBank(up, down, 2)
    ids, wt = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    z, lp = torch.zeros(4, 100), torch.zeros(4, 2)
    saved = fq.DistillLoss(torch.zeros(4), torch.zeros(4, 7))
    for call in [
        lambda: fq.fp4_gemm_epilogue(a, w), lambda: fq.fp4_wo_gemm_epilogue(x, w), lambda: fq.fp4_epilogue_backward(y, y, "silu"),
        lambda: fq.fp4_moe_route(z, 2), lambda: fq.fp4_moe(x, bank, ids, wt), lambda: fq.fp4_distill_loss(z, ids, lp),
        lambda: fq.fp4_distill_loss_backward(z, ids, lp, saved, torch.zeros(4)),                             # host tensors
        lambda: fq.fp4_gemm_epilogue(a, w, act="swish"), lambda: fq.fp4_gemm_epilogue(a, w, bias=b[:63]),
        lambda: fq.fp4_gemm_epilogue(a, w, bias=b.half()), lambda: fq.fp4_gemm_epilogue(a, w, mul=y.float()),
        lambda: fq.fp4_gemm_epilogue(a, w, residual=y[:3]), lambda: fq.fp4_gemm_epilogue(a, w, mul=y.t()),
        lambda: fq.fp4_wo_gemm_epilogue(x.float(), w), lambda: fq.fp4_wo_gemm_epilogue(x[:, :128], w),
        lambda: fq.fp4_epilogue_backward(y.float(), y), lambda: fq.fp4_epilogue_backward(y, None, "silu"),
        lambda: fq.fp4_epilogue_backward(y, y[:, :8], "silu"), lambda: fq.fp4_epilogue_backward(y, y, mul=y.float()),
        lambda: fq.fp4_moe_route(z.half(), 2), lambda: fq.fp4_moe_route(z, 2, score="top"), lambda: fq.fp4_moe_route(z, 2, bias=torch.zeros(99)),
        lambda: fq.fp4_moe(x, fq.MoeBank(up, down, 3), ids, wt), lambda: fq.fp4_moe(x, fq.MoeBank(down, up, 2), ids, wt),
        lambda: fq.fp4_moe(x, fq.MoeBank(up, down, 2, up_scale=torch.ones(3)), ids, wt), lambda: fq.fp4_moe(x.float(), bank, ids, wt),
        lambda: fq.fp4_moe(x, bank, ids.long(), wt), lambda: fq.fp4_moe(x, bank, ids, wt.to(bf)), lambda: fq.fp4_moe(x, bank, ids[:3], wt[:3]),
        lambda: fq.fp4_moe(x, bank, ids, wt[:, :1]), lambda: fq.fp4_moe(x, bank, ids, wt, act="tanh"),
        lambda: fq.fp4_moe(x, bank, ids, wt, residual=x.float()),
        lambda: fq.fp4_distill_loss(z.half(), ids, lp), lambda: fq.fp4_distill_loss(z, ids.long(), lp), lambda: fq.fp4_distill_loss(z, ids, lp[:, :1]),
        lambda: fq.fp4_distill_loss(z, ids, lp, rest="tail"), lambda: fq.fp4_distill_loss(z[:3], ids, lp),
        lambda: fq.fp4_distill_loss_backward(z, ids, lp, saved, torch.zeros(3)),
        lambda: fq.fp4_distill_loss_backward(z, ids, lp, fq.DistillLoss(saved.loss, saved.stats[:, :6]), torch.zeros(4)),
    ]:
        with pytest.raises(ValueError):
            call()
