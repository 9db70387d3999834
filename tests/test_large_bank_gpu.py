"""A bank of as many adapters as the calls take, each with a long K: more
64 x 64 tiles than one dimension of a launch may have work groups."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
BF = torch.bfloat16


def test_backward_of_many_long_adapters():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    la, r, k, n, m = 16384, 8, 65536, 8, 72
    assert la * (k // 64) * 256 >= 2 ** 32 and m * k > 2 ** 22
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = torch.zeros(la, r, k, dtype=BF, device="cuda"), torch.zeros(la, n, r, dtype=BF, device="cuda")
    used = torch.tensor([0, 5, la - 1], device="cuda")
    a[used] = torch.randint(-2, 3, (3, r, k), generator=g, device="cuda").to(BF)
    b[used] = torch.randint(-2, 3, (3, n, r), generator=g, device="cuda").to(BF)
    # whole numbers of a few bits: every sum is exact, in any order
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").to(BF)
    dy = torch.randint(-1, 2, (m, n), generator=g, device="cuda").to(BF)
    t = torch.randint(-4, 5, (m, r), generator=g, device="cuda").float()
    slots = used[torch.arange(m, device="cuda") % 3].int()
    dx, da, db = fq.fp4_lora_backward(dy, x, t, fq.LoraBank(a, b, torch.ones(la, device="cuda")), slots, grad_dtype=torch.float32)
    for i, l in enumerate(used.tolist()):
        at = torch.arange(i, m, 3, device="cuda")
        dt = dy[at].float() @ b[l].float()
        assert torch.equal(dx[at].float(), (dt @ a[l].float()).to(BF).float())
        assert torch.equal(da[l], dt.t().contiguous() @ x[at].float())
        assert torch.equal(db[l], dy[at].float().t().contiguous() @ t[at])
        da[l] = 0
    assert not da.view(la, -1).any()
