"""The entropy's gradient on confident rows, where it is a difference of small
numbers and needs all of binary32."""
import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
F = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("lead", [8.0, 12.0, 16.0, 20.0, 30.0])
@pytest.mark.parametrize("v", [1000, 9000])
def test_entropy_gradient_of_a_confident_row(lead, v):
    """One logit leads, so its log p and the entropy are small, and its
    gradient -p (log p + H) is their sum.  In it log s, which H contains, meets
    the -log s of log p: both are the same binary32 number (rounded against 1:
    2^-24 of s), so what is left is off by the relative error of w = sum e d.
    That is 6e-6 of the powers, 3 roundings of d, and 2 x 256 roundings of the
    sums at the most (v / 256 terms a thread, then joined): below 4e-5.  To it
    come 2^-22 of the magnitudes |log p|, H and log s, and a step of p."""
    g = torch.Generator().manual_seed(int(lead))
    z = torch.randn(4, v, generator=g)
    at = torch.tensor([0, v // 3, v // 2, v - 1])
    z[torch.arange(4), at] = lead
    zd = z.cuda()
    f = fq.fp4_token_logprobs(zd)
    dz = fq.fp4_token_logprobs_backward(zd, None, f, grad_entropy=torch.ones(4, device="cuda")).cpu().to(F)
    d = z.to(F) - z.to(F).amax(-1, keepdim=True)
    logs = d.exp().sum(-1, keepdim=True).log()
    lp = d - logs
    p = lp.exp()
    ent = -(p * lp).sum(-1, keepdim=True)
    want = -p * (lp + ent)
    tol = p * (4e-5 * (lp + ent).abs() + 2.0 ** -22 * (lp.abs() + ent + logs) + 4e-5 * ent) + 2.0 ** -22 * want.abs() + 1e-37
    off = (dz - want).abs()
    assert not (~(off <= tol)).any(), (float((off / tol).max()), (~(off <= tol)).nonzero()[0].tolist())
