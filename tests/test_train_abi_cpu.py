"""Host-side checks of the adapter, token-probability and residual-norm calls
that need no GPU: invalid arguments are refused before any launch (the
pointers are never dereferenced), workspaces have the sizes the calls ask
for, and the binding refuses what does not fit the kernels."""
import ctypes

import pytest
import torch

import fp4_block_scaled_quantize_amd as fq

FAKE = 0x10000      # 16-byte aligned, never dereferenced: validation fails first
ROOM = 1 << 40


def _bank(a=FAKE, b=FAKE, scale=FAKE, adapters=2, rank=16, k=256, n=64):
    return fq.Fp4LoraBankC(a, b, scale, adapters, rank, k, n)


def _apply(bank=None, x=FAKE, ldx=256, m=32, slots=FAKE, base=None, ldb=64, y=FAKE, ldy=64, t=FAKE, ws=FAKE, room=ROOM):
    bank = bank or _bank()
    return fq.lib().fp4_lora_apply(x, ldx, m, ctypes.byref(bank), slots, base, ldb, y, ldy, t, ws, room, None)


@pytest.mark.parametrize("kw,want", [
    (dict(bank=_bank(a=None)), -1), (dict(bank=_bank(b=None)), -1), (dict(bank=_bank(scale=None)), -1),
    (dict(bank=_bank(adapters=0)), -3), (dict(bank=_bank(rank=0)), -3), (dict(bank=_bank(rank=12)), -3),
    (dict(bank=_bank(k=250)), -3), (dict(bank=_bank(n=60)), -3), (dict(bank=_bank(rank=136)), -2),
    (dict(bank=_bank(adapters=16385)), -2), (dict(bank=_bank(a=FAKE + 8)), -4), (dict(bank=_bank(b=FAKE + 2)), -4),
    (dict(m=-1), -3), (dict(m=(1 << 20) + 1), -2), (dict(slots=None), -1), (dict(slots=FAKE + 2), -4),
    (dict(x=None), -1), (dict(ldx=248), -3), (dict(ldx=260), -4), (dict(x=FAKE + 8), -4), (dict(ldx=1 << 38), -2),
    (dict(y=None), -1), (dict(ldy=56), -3), (dict(y=FAKE + 4), -4), (dict(base=FAKE + 8), -4), (dict(base=FAKE, ldb=72), -3),
    (dict(t=None), -1), (dict(t=FAKE + 4), -4), (dict(ws=None), -1), (dict(room=15), -1), (dict(ws=FAKE + 8), -4),
])
def test_apply_rejects_before_launch(kw, want):
    # a long K is taken in ranges, which need a workspace, so that its checks are reached
    if "bank" not in kw:
        k = 65536
        kw = dict(kw, bank=_bank(k=k), ldx=kw.get("ldx", k) if kw.get("ldx") not in (248, 260) else kw["ldx"] + k - 256)
    assert _apply(**kw) == want


def test_apply_refuses_no_bank():
    assert fq.lib().fp4_lora_apply(FAKE, 256, 4, None, FAKE, None, 0, FAKE, 64, FAKE, FAKE, ROOM, None) == -1


def _backward(m=32, dy=FAKE, ldd=64, x=FAKE, ldx=256, t=FAKE, dxb=None, ldxb=256, dx=FAKE + 64, lddx=256, da=FAKE, db=FAKE,
              gd=0, ws=FAKE, room=ROOM, slots=FAKE):
    return fq.lib().fp4_lora_backward(dy, ldd, x, ldx, m, t, ctypes.byref(_bank()), slots, dxb, ldxb, dx, lddx, da, db, gd,
                                      ws, room, None)


@pytest.mark.parametrize("kw,want", [
    (dict(gd=2), -1), (dict(m=-1), -3), (dict(slots=None), -1), (dict(dy=None), -1), (dict(ldd=56), -3),
    (dict(dy=FAKE + 8), -4), (dict(x=None), -1), (dict(ldx=255), -3), (dict(dx=None), -1), (dict(lddx=260), -4),
    (dict(dxb=FAKE + 8), -4), (dict(dxb=FAKE + 64, ldxb=264), -3), (dict(dx=FAKE), -1), (dict(dx=FAKE, x=FAKE + 32), -1), (dict(t=None), -1), (dict(da=None), -1), (dict(db=None), -1),
    (dict(da=FAKE + 8), -4), (dict(ws=None), -1), (dict(room=100), -1), (dict(ws=FAKE + 8), -4),
])
def test_backward_rejects_before_launch(kw, want):
    assert _backward(**kw) == want


def test_lora_workspace():
    ws = fq.lib().fp4_lora_workspace
    assert ws(3, 1, 8, 8, 8, 1) == -1 and ws(0, -1, 8, 8, 8, 1) == -3 and ws(0, 1, 0, 8, 8, 1) == -3
    assert ws(0, (1 << 20) + 1, 8, 8, 8, 1) == -2 and ws(0, 1, 8, 8, 136, 1) == -2
    assert ws(0, 8192 * 4, 4096, 4096, 16, 1) == 0         # rows alone fill the device: T needs no partial sums
    assert ws(2, 1, 64, 256, 16, 1) >= 4 * 16
    for m in (0, 1, 7, 16, 17, 64, 500, 8192):
        for call in (0, 1, 2):
            b = ws(call, m, 11008, 4096, 16, 4)
            assert b >= 0 and b % 16 == 0
            # partial sums are bounded: at most 32 of T and 16 of the gradients, and B, A once more
            assert b <= 4 * 33 * m * 16 + 4 * 16 * (11008 + 4096) * 17 * 4 + 4096


def test_wo_gemm_lora_rejects_before_launch():
    L = fq.lib()
    w = fq.Fp4TensorC(FAKE, FAKE, FAKE, 64, 256, fq.Fp4Format(16, 0, 0, 1))

    def call(bank, m=4, w=w, slots=FAKE, ws=FAKE, room=ROOM):
        return L.fp4_wo_gemm_lora(FAKE, 256, m, ctypes.byref(w), ctypes.byref(bank), slots, FAKE, 64, ws, room, None)
    assert call(_bank(), m=0) == -2 and call(_bank(), m=17) == -2
    assert call(_bank(n=56)) == -3 and call(_bank(k=512)) == -3 and call(_bank(rank=4)) == -3
    assert call(_bank(), slots=None) == -1 and call(_bank(), ws=None) == -1 and call(_bank(), room=8) == -1
    none = fq.Fp4TensorC(FAKE, FAKE, FAKE, 0, 256, fq.Fp4Format(16, 0, 0, 1))
    assert call(_bank(), w=none) == -3
    w2 = fq.Fp4TensorC(FAKE, FAKE, FAKE, 64, 256, fq.Fp4Format(16, 0, 0, 1, 1, 5))
    assert call(_bank(), w=w2) == -2                       # a transformed weight


def _lp(z=FAKE, dt=1, ld=1000, n=4, v=1000, tok=FAKE, temp=1.0, top=3, lp=FAKE, ent=FAKE, st=FAKE, ids=FAKE, best=FAKE,
        ws=FAKE, room=ROOM):
    return fq.lib().fp4_token_logprobs(z, dt, ld, n, v, tok, temp, top, lp, ent, st, ids, best, ws, room, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), -1), (dict(temp=0.0), -1), (dict(temp=-1.0), -1), (dict(temp=float("nan")), -1),
    (dict(temp=float("inf")), -1), (dict(temp=1e-45), -1), (dict(temp=4e-39), -1), (dict(n=-1), -3), (dict(v=0), -3), (dict(ld=999), -3),
    (dict(v=1 << 27, ld=1 << 27), -2), (dict(n=1 << 22), -2), (dict(z=None), -1), (dict(z=FAKE + 1), -4), (dict(dt=0, z=FAKE + 2), -4),
    (dict(top=-1), -2), (dict(top=33), -2), (dict(v=2, ld=2), -3), (dict(ent=None), -1), (dict(st=None), -1),
    (dict(lp=None), -1), (dict(ids=None), -1), (dict(best=None), -1), (dict(tok=FAKE + 4), -4), (dict(ent=FAKE + 2), -4),
    (dict(v=20000, ld=20000, ws=None), -1), (dict(v=20000, ld=20000, room=8), -1),
])
def test_logprobs_rejects_before_launch(kw, want):
    assert _lp(**kw) == want


def test_logprobs_workspace():
    ws = fq.lib().fp4_token_logprobs_workspace
    assert ws(-1, 5, 0) == -3 and ws(1, 0, 0) == -3 and ws(1, 5, 33) == -2
    assert ws(0, 128000, 5) == 0 and ws(1, 1000, 5) == 0 and ws(512, 128000, 5) == 0
    assert 0 < ws(1, 128000, 20) <= 64 * (16 + 160)
    assert 0 < ws(300, 128000, 32) <= 300 * 64 * (16 + 256)


def test_logprobs_backward_rejects_before_launch():
    def call(z=FAKE, ld=100, tok=FAKE, ent=FAKE, st=FAKE, gl=FAKE, ge=FAKE, d=FAKE + 64, ldd=100, temp=1.0):
        return fq.lib().fp4_token_logprobs_backward(z, 0, ld, 4, 100, tok, temp, ent, st, gl, ge, d, ldd, None)
    assert call(z=None) == -1 and call(ent=None) == -1 and call(st=None) == -1 and call(d=None) == -1
    assert call(tok=None) == -1 and call(temp=0.0) == -1
    assert call(ldd=99) == -3 and call(d=FAKE, ldd=104) == -3
    assert call(d=FAKE + 2) == -4 and call(gl=FAKE + 2) == -4


def _norm(x=FAKE, ldx=64, r=FAKE, ldr=64, rows=4, cols=64, w2=FAKE, w1=None, gate=None, alpha=1.0, eps=1e-6, xd=1, rd=0, wd=1):
    return fq.Fp4NormC(x, ldx, r, ldr, rows, cols, w2, w1, gate, alpha, eps, xd, rd, wd)


@pytest.mark.parametrize("kw,want", [
    (dict(xd=3), -1), (dict(rd=-1), -1), (dict(wd=2), -1), (dict(alpha=float("nan")), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("inf")), -1), (dict(rows=-1), -3), (dict(cols=0), -3), (dict(cols=32769, ldx=40000, ldr=40000), -2), (dict(rows=1 << 22), -2),
    (dict(w2=None), -1), (dict(x=None), -1), (dict(r=None), -1), (dict(ldx=63), -3), (dict(ldr=63), -3),
    (dict(x=FAKE + 1), -4), (dict(r=FAKE + 2), -4), (dict(w1=FAKE + 1), -4), (dict(gate=FAKE + 2), -4),
])
def test_norm_rejects_before_launch(kw, want):
    L, a = fq.lib(), _norm(**kw)
    c = max(a.cols, 1)
    assert L.fp4_residual_norm(ctypes.byref(a), FAKE, c, FAKE, c, FAKE, None) == want
    assert L.fp4_residual_norm_backward(ctypes.byref(a), FAKE, FAKE, c, FAKE, c, FAKE, c, FAKE, c, FAKE, FAKE, FAKE, FAKE,
                                        ROOM, None) == want


def test_norm_output_checks():
    L = fq.lib()
    a = _norm(w1=FAKE, gate=FAKE)

    def fwd(h=FAKE, ldh=64, n=FAKE + 64, ldn=64, st=FAKE):
        return L.fp4_residual_norm(ctypes.byref(a), h, ldh, n, ldn, st, None)

    def back(st=FAKE, dx=FAKE + 64, lddx=64, dr=FAKE + 64, dw2=FAKE, dw1=FAKE, dg=FAKE, ws=FAKE, room=ROOM, lddn=64):
        return L.fp4_residual_norm_backward(ctypes.byref(a), st, FAKE, lddn, FAKE, 64, dx, lddx, dr, 64, dw2, dw1, dg, ws,
                                            room, None)
    assert L.fp4_residual_norm(None, FAKE, 64, FAKE, 64, FAKE, None) == -1
    assert fwd(h=None) == -1 and fwd(n=None) == -1 and fwd(st=None) == -1 and fwd(ldh=63) == -3 and fwd(h=FAKE + 2) == -4
    assert fwd(h=FAKE, ldh=72) == -3                       # in place with another stride
    for kw in (dict(st=None), dict(dx=None), dict(dr=None), dict(dw2=None), dict(dw1=None), dict(dg=None), dict(ws=None),
               dict(room=16)):
        assert back(**kw) == -1, kw
    assert back(lddn=63) == -3 and back(dx=FAKE, lddx=72) == -3 and back(ws=FAKE + 4) == -4 and back(dw2=FAKE + 2) == -4
    need = L.fp4_residual_norm_workspace
    assert need(-1, 8, 0) == -3 and need(1, 0, 0) == -3 and need(1, 32769, 0) == -2
    assert need(0, 64, 1) >= 2 * 64 * 4 and need(100000, 64, 0) <= 1024 * 64 * 4


class _NoCalls:
    """Stands in for the library: any call is a test failure."""
    def __getattr__(self, name):
        raise AssertionError(f"library function {name} reached")


def test_binding_checks_before_any_call(monkeypatch):
    monkeypatch.setattr(fq, "lib", lambda: _NoCalls())
    bf = torch.bfloat16
    x, s = torch.zeros(4, 256, dtype=bf), torch.zeros(4, dtype=torch.int32)
    bank = fq.LoraBank(torch.zeros(2, 16, 256, dtype=bf), torch.zeros(2, 64, 16, dtype=bf), torch.ones(2))
    w = fq.QTensor.empty(64, 256, 16, "e4m3", device="cpu")
    t, dy = torch.zeros(4, 16), torch.zeros(4, 64, dtype=bf)
    z, tok = torch.zeros(4, 100), torch.zeros(4, dtype=torch.long)
    saved = fq.TokenLogprobs(torch.zeros(4), torch.zeros(4), torch.zeros(4, 2), None, None)
    wt = torch.ones(256)
    calls = [
        lambda: fq.fp4_lora_apply(x, bank, s), lambda: fq.fp4_wo_gemm_lora(x, w, bank, s),        # host tensors
        lambda: fq.fp4_lora_backward(dy, x, t, bank, s), lambda: fq.fp4_token_logprobs(z, tok),
        lambda: fq.fp4_token_logprobs_backward(z, tok, saved, torch.zeros(4)),
        lambda: fq.fp4_residual_norm(x, x, wt), lambda: fq.fp4_residual_norm_backward(x, x, x, x, wt, torch.zeros(4, 2)),
        lambda: fq.fp4_lora_apply(x.float(), bank, s), lambda: fq.fp4_lora_apply(x[:, :128], bank, s),
        lambda: fq.fp4_lora_apply(x, bank, s.long()), lambda: fq.fp4_lora_apply(x, bank, s[:3]),
        lambda: fq.fp4_lora_apply(x, fq.LoraBank(bank.a, bank.b[:1], bank.scale), s),
        lambda: fq.fp4_lora_apply(x, fq.LoraBank(bank.a.float(), bank.b, bank.scale), s),
        lambda: fq.fp4_lora_apply(x, fq.LoraBank(bank.a, bank.b.transpose(1, 2), bank.scale), s),
        lambda: fq.fp4_lora_backward(dy.float(), x, t, bank, s), lambda: fq.fp4_lora_backward(dy, x, t[:, :8], bank, s),
        lambda: fq.fp4_lora_backward(dy, x, t, bank, s, grad_dtype=torch.float16),
        lambda: fq.fp4_token_logprobs(z.half(), tok), lambda: fq.fp4_token_logprobs(z, tok.int()),
        lambda: fq.fp4_token_logprobs(z.t(), tok), lambda: fq.fp4_token_logprobs(z, tok[:2]),
        lambda: fq.fp4_token_logprobs_backward(z, None, saved, torch.zeros(4)),
        lambda: fq.fp4_token_logprobs_backward(z, tok, saved, torch.zeros(4, dtype=torch.float64)),
        lambda: fq.fp4_residual_norm(x, x[:3], wt), lambda: fq.fp4_residual_norm(x, x, wt[:8]),
        lambda: fq.fp4_residual_norm(x, x, wt, w_post=wt.to(bf)), lambda: fq.fp4_residual_norm(x, x, wt, gate=wt),
        lambda: fq.fp4_residual_norm_backward(x.float(), x, x, x, wt, torch.zeros(4, 2)),
        lambda: fq.fp4_residual_norm_backward(x, x, x, x, wt, torch.zeros(4)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            print("call", i)
