"""The intermediates T and dT of the adapter calls keep binary32's 24 bits
where they enter the second product, whatever the type of its result.

Every sum here is exact in binary32: T (or dT) holds 1 + 2^-10 + 2^-20 in one
rank and 1 + 2^-10 in another, and the second product subtracts the two.  So
the result is a scale times 2^-20 exactly, and any rounding of T to fewer than
21 bits loses it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
BF = torch.bfloat16
PARTS = (1.0, 2.0 ** -5, 2.0 ** -10)      # their squares add up to 1 + 2^-10 + 2^-20


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bank(la, n, k, r, at):
    """A's ranks 0 and r - 1 take PARTS, and PARTS without its last, at `at`
    along K; B's are 1 and -1 everywhere."""
    a, b = torch.zeros(la, r, k), torch.zeros(la, n, r)
    a[:, 0, at], a[:, r - 1, at] = torch.tensor(PARTS), torch.tensor([*PARTS[:2], 0.0])
    b[:, :, 0], b[:, :, r - 1] = 1.0, -1.0
    return a.to(BF), b.to(BF), torch.arange(la) + 1.0


def _slots(m, la):
    return torch.arange(m).mul(la).div(m, rounding_mode="floor").int()


SHAPES = [(1, 72, 264, 8, 1), (16, 136, 520, 96, 3), (40, 264, 264, 16, 2), (130, 136, 264, 48, 3), (200, 264, 136, 128, 2),
          (2100, 136, 2056, 24, 3)]


@pytest.mark.parametrize("m,n,k,r,la", SHAPES)
def test_apply(m, n, k, r, la):
    at = [3, k // 2, k - 1]
    a, b, sc = _bank(la, n, k, r, at)
    x = torch.zeros(m, k)
    x[:, at] = torch.tensor(PARTS)
    slots = _slots(m, la)
    y, t = fq.fp4_lora_apply(x.to(BF).cuda(), fq.LoraBank(a.cuda(), b.cuda(), sc.cuda()), slots.cuda())
    assert (t[:, 0] == 1 + 2.0 ** -10 + 2.0 ** -20).all() and (t[:, r - 1] == 1 + 2.0 ** -10).all()
    assert torch.equal(y.cpu().float(), (sc[slots.long()] * 2.0 ** -20)[:, None].expand(m, n))


@pytest.mark.parametrize("m,n,k,r,la", SHAPES)
@pytest.mark.parametrize("gdt", [torch.float32, BF])
def test_backward(m, n, k, r, la, gdt):
    """dT from PARTS along N; dx subtracts its two ranks.  Two neighbouring
    rows of an adapter, one with the third part and one without, subtract in dA
    (x of opposite sign) and in dB (dy of opposite sign)."""
    at = [1, n // 2, n - 1]
    bt, at_, sc = _bank(la, k, n, r, at)                     # the bank's roles exchanged: B along N like A along K
    a, b = at_.transpose(1, 2).contiguous(), bt.transpose(1, 2).contiguous()
    dy, x = torch.zeros(m, n), torch.zeros(m, k)
    dy[:, at] = torch.tensor(PARTS)
    slots = _slots(m, la)
    bank = fq.LoraBank(a.cuda(), b.cuda(), sc.cuda())
    t = torch.zeros(m, r)
    dx, _, _ = fq.fp4_lora_backward(dy.to(BF).cuda(), x.to(BF).cuda(), t.cuda(), bank, slots.cuda(), grad_dtype=gdt)
    assert torch.equal(dx.cpu().float(), (sc[slots.long()] * 2.0 ** -20)[:, None].expand(m, k))
    if m < 2:
        return
    # dA: rows 0 and 1 of adapter 0
    dy[1, at[2]] = 0.0
    x[0], x[1] = 1.0, -1.0
    t[0], t[1] = 1 + 2.0 ** -10 + 2.0 ** -20, -(1 + 2.0 ** -10)
    one = torch.zeros(m, dtype=torch.int32)
    _, da, _ = fq.fp4_lora_backward(dy.to(BF).cuda(), x.to(BF).cuda(), t.cuda(), bank, one.cuda(), grad_dtype=gdt)
    assert (da[0, 0].float() == 2.0 ** -20).all()
    # dB: the same two rows with equal dy
    dy[1] = dy[0] = 1.0
    dy[2:] = 0.0
    _, _, db = fq.fp4_lora_backward(dy.to(BF).cuda(), x.to(BF).cuda(), t.cuda(), bank, one.cuda(), grad_dtype=gdt)
    assert (db[0].float() == 2.0 ** -20).all()
