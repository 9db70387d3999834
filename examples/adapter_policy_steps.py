"""Policy-gradient steps of low-rank adapters over FP4 weights, and a rollout
step that serves several requests' adapters at once (quant_prune_distill/574:
NVFP4 weight-only rollouts, adapters trained by reinforcement learning).

One residual block between two norms and a vocabulary head, all weights in
FP4, the adapters of two tasks in bf16:

    n  = RMSNorm(r) w_in
    y  = n W^T + s_a (n A_a^T) B_a^T          FP4 product, adapter of each row's task
    r' = alpha r + gate RMSNorm(y) w_post,  m = RMSNorm(r') w_pre
    z  = m H^T                                FP4 product
    loss = sum(-advantage log p(token) - 0.01 entropy) / rows

Run: python examples/adapter_policy_steps.py   (needs the GPU library built)
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp4_block_scaled_quantize_amd as fq  # noqa: E402


class Block:
    def __init__(self, hidden=512, vocab=2048, rank=16, tasks=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, sd, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device="cuda") * sd).to(dtype)

        w, head = normal(hidden, hidden, sd=hidden ** -0.5), normal(vocab, hidden, sd=hidden ** -0.5)
        # each weight in both orientations: along its inputs for the forward
        # product, along its outputs for the gradient's
        self.w, self.w_t = fq.fp4_quantize_both(w)
        self.head, self.head_t = fq.fp4_quantize_both(head)
        self.bank = fq.LoraBank(normal(tasks, rank, hidden, sd=hidden ** -0.5), normal(tasks, hidden, rank, sd=0.01),
                                torch.full((tasks,), 2.0, device="cuda"))
        self.w_in, self.w_pre, self.w_post = (1 + normal(hidden, sd=0.05, dtype=torch.float32) for _ in range(3))
        self.alpha = 0.8

    def forward(self, r, task, gate):
        """Logits of the rows, and what the backward pass reads."""
        none = torch.zeros_like(r)
        _, n, s_in = fq.fp4_residual_norm(none, r, self.w_in)                  # the first norm: nothing to add yet
        y, t = fq.fp4_lora_apply(n, self.bank, task, base=fq.fp4_gemm(fq.fp4_quantize(n), self.w))
        _, m, s_mid = fq.fp4_residual_norm(y, r, self.w_pre, w_post=self.w_post, gate=gate, alpha=self.alpha)
        z = fq.fp4_gemm(fq.fp4_quantize(m), self.head)
        return z, (none, n, s_in, y, t, s_mid)

    def backward(self, dz, saved, r, task, gate):
        """Gradients of the adapters, the norms' weights and the residual stream."""
        none, n, s_in, y, t, s_mid = saved
        dm = fq.fp4_gemm(fq.fp4_quantize(dz, rounding="stochastic", seed=1), self.head_t)
        g = fq.fp4_residual_norm_backward(dm, None, y, r, self.w_pre, s_mid, w_post=self.w_post, gate=gate,
                                          alpha=self.alpha)
        dn = fq.fp4_gemm(fq.fp4_quantize(g.dx, rounding="stochastic", seed=2), self.w_t)
        dn, da, db = fq.fp4_lora_backward(g.dx, n, t, self.bank, task, dx_base=dn, dx=dn)
        first = fq.fp4_residual_norm_backward(dn, g.dres, none, r, self.w_in, s_in)
        return da, db, (first.dw_pre, g.dw_pre, g.dw_post), first.dres


def train(block, steps=8, rows=256, rate=0.5, seed=1):
    """The loss and the mean advantage-weighted log probability of each step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    hidden, vocab, tasks = block.w.cols, block.head.rows, block.bank.a.shape[0]
    r = torch.randn(rows, hidden, generator=g, device="cuda").bfloat16()
    task = torch.arange(rows, device="cuda").mul(tasks).div(rows, rounding_mode="floor").int()
    task[::17] = -1                                                            # rows of the base model
    gate = torch.rand(rows, generator=g, device="cuda") + 0.5
    token = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    token[::13] = -100                                                         # padding
    advantage = torch.rand(rows, generator=g, device="cuda") + 0.5
    history = []
    for _ in range(steps):
        z, saved = block.forward(r, task, gate)
        f = fq.fp4_token_logprobs(z, token)
        history.append((-(advantage * f.logprob) - 0.01 * f.entropy).sum().div(rows).item())
        dz = fq.fp4_token_logprobs_backward(z, token, f, -advantage / rows, torch.full_like(advantage, -0.01 / rows))
        da, db, _, _ = block.backward(dz, saved, r, task, gate)
        block.bank.a -= (rate * da).to(torch.bfloat16)
        block.bank.b -= (rate * db).to(torch.bfloat16)
    return history


def rollout(block, requests=8, tokens=4, seed=2):
    """A few greedy steps of a batch whose requests use different adapters:
    the weight-only products with the adapters in their epilogue, the norms and
    the chosen tokens' log probabilities with their alternatives."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    hidden, tasks = block.w.cols, block.bank.a.shape[0]
    embed = torch.randn(block.head.rows, hidden, generator=g, device="cuda").bfloat16()
    r = torch.randn(requests, hidden, generator=g, device="cuda").bfloat16()
    task = (torch.arange(requests, device="cuda") % (tasks + 1) - 1).int()     # -1: the base model
    out = []
    for _ in range(tokens):
        _, n, _ = fq.fp4_residual_norm(torch.zeros_like(r), r, block.w_in)
        y = fq.fp4_wo_gemm_lora(n, block.w, block.bank, task)
        _, m, _ = fq.fp4_residual_norm(y, r, block.w_pre, w_post=block.w_post, alpha=block.alpha)
        f = fq.fp4_token_logprobs(fq.fp4_wo_gemm(m, block.head), top=4)
        out.append((f.top_ids, f.top_logprobs, f.entropy))
        r = embed[f.top_ids[:, 0].long()]
    return out


if __name__ == "__main__":
    model = Block()
    for i, loss in enumerate(train(model)):
        print(f"step {i}: loss {loss:.4f}")
    ids, logprobs, entropy = rollout(model)[0]
    for i in range(ids.shape[0]):
        print(f"request {i}: tokens {ids[i].tolist()} log p {[round(v, 3) for v in logprobs[i].tolist()]} "
              f"entropy {entropy[i].item():.3f}")
