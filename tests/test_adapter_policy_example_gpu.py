"""The example runs the adapter, token-probability and norm calls together
with the FP4 products: the loss falls, and the adapters' gradients agree with
the same step taken in binary64 from the dequantized weights as far as the FP4
rounding of activations and gradients lets them."""
import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

fq = pytest.importorskip("fp4_block_scaled_quantize_amd")


@pytest.fixture
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("adapter_policy_steps", os.path.join(ROOT, "examples", "adapter_policy_steps.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_policy_steps_lower_the_loss(example):
    history = example.train(example.Block(), steps=6)
    assert all(b < a for a, b in zip(history, history[1:])), history


def test_rollout_serves_each_request_its_adapter(example):
    block = example.Block()
    out = example.rollout(block, requests=7, tokens=2)
    ids, logprobs, entropy = out[0]
    assert ids.shape == (7, 4) and torch.isfinite(logprobs).all() and (entropy > 0).all()
    assert (logprobs[:, :-1] >= logprobs[:, 1:]).all()
    # a request of the base model (adapter -1) sees no adapter at all
    block.bank.b.zero_()
    again = example.rollout(block, requests=7, tokens=1)[0]
    base = torch.arange(7) % 3 == 0
    assert torch.equal(again[0].cpu()[base], ids.cpu()[base]) and torch.equal(again[1].cpu()[base], logprobs.cpu()[base])


def test_gradients_point_along_the_exact_ones(example):
    block = example.Block(hidden=256, vocab=512)
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = 128
    r = torch.randn(rows, 256, generator=g, device="cuda").bfloat16()
    task = (torch.arange(rows, device="cuda") % 2).int()
    gate = torch.rand(rows, generator=g, device="cuda") + 0.5
    token = torch.randint(0, 512, (rows,), generator=g, device="cuda")
    z, saved = block.forward(r, task, gate)
    f = fq.fp4_token_logprobs(z, token)
    ones = torch.full((rows,), -1.0 / rows, device="cuda")
    da, db, _, _ = block.backward(fq.fp4_token_logprobs_backward(z, token, f, ones), saved, r, task, gate)

    def norm(v):
        return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt()

    d = lambda q: fq.fp4_dequantize(q).double()            # noqa: E731
    a, b = (v.double().requires_grad_() for v in (block.bank.a, block.bank.b))
    n = norm(r.double()) * block.w_in.double()
    idx = task.long()
    t = torch.stack([n @ a[i].t() for i in range(2)])[idx, torch.arange(rows, device="cuda")]
    delta = torch.stack([t @ b[i].t() for i in range(2)])[idx, torch.arange(rows, device="cuda")]
    y = n @ d(block.w).t() + 2.0 * delta
    h = block.alpha * r.double() + gate.double()[:, None] * norm(y) * block.w_post.double()
    lp = torch.log_softmax((norm(h) * block.w_pre.double()) @ d(block.head).t(), -1)
    (-lp[torch.arange(rows, device="cuda"), token].mean()).backward()
    for got, want in ((da, a.grad), (db, b.grad)):
        cos = torch.nn.functional.cosine_similarity(got.double().flatten(), want.flatten(), dim=0)
        assert cos > 0.9, float(cos)                       # four-bit activations and gradients lie between
