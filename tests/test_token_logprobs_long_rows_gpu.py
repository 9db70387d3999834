"""The sums of long rows, whose threads add thousands of terms each."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")
F = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("top", [1, 0])
@pytest.mark.parametrize("dtype,n,v", [(torch.bfloat16, 2001, 1 << 19), (torch.float32, 2001, 1 << 18)])
def test_sums_of_long_rows(dtype, n, v, top):
    """Rows whose first logits are zeros (every thread then sums about zero)
    and all others one lower value: equal terms, whose roundings in a sum all
    go one way while the sum stays in a binade.  A thread's sum may take 32
    roundings for the terms of a round of loads, one for each round (v / 2048 of
    bf16, v / 1024 of binary32 in one wave) and 8 in the joins: 296 x 2^-24 =
    1.8e-5.  With the terms' own 2^-22, and 3 roundings of d (|d| < 5), it is
    below 3e-5 of s and of w = sum e d.  log s is off by that, w / s by twice
    that of itself; 2^-22 of log v comes to them."""
    low = torch.linspace(0.25, 3.0, n).to(dtype)
    z = (-low).cuda()[:, None].expand(n, v).contiguous()
    head = 2048
    z[:, :head] = 0.0
    tok = torch.full((n,), 7, dtype=torch.long, device="cuda")
    f = fq.fp4_token_logprobs(z, tok, top=top)
    d = -low.to(F)
    s = head + (v - head) * d.exp()
    mean = (v - head) * d.exp() * d / s
    for got, want, tol in ((f.logprob, -s.log(), 3e-5 + 0 * s), (f.entropy, s.log() - mean, 3e-5 * (1 + 2 * mean.abs()))):
        off = (got.cpu().to(F) - want).abs()
        worst = (off - tol).argmax()
        assert (off <= tol + math.log(v) * 2.0 ** -22).all(), (float(off[worst]), float(tol[worst]), float(low[worst]))
