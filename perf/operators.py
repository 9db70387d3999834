"""Cases of the adapter, token-probability and residual-norm operators.

Every case is one call, or one forward and backward pair, as a program that
fine-tunes low-rank adapters over FP4 weights with a policy gradient makes
it.  `run` computes it from elementary torch operations in binary32 (rounded
once, at the end) or, where `own` is set, through the package's entry points;
`exact` computes it in binary64.

Kinds of a case:
  decode     y = x W^T + s_a (x A_a^T) B_a^T for at most 16 rows, W in FP4, each row with the adapter of its request
  apply      y = base + s_a (x A_a^T) B_a^T for any number of rows (base: the shared projection's output)
  backward   the gradients of `apply` with respect to x, A and B
  logprobs   log probability of a given token, entropy and the top alternatives of each row of logits
  policy     `logprobs` and the gradient of a policy loss with respect to the logits
  norm       h = alpha r + gate RMSNorm(x) w_post and n = RMSNorm(h) w_pre
  norm_step  `norm` and its gradients
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one request being generated: the up projection of a decoder layer, one token
        dict(name="decode 1 row", kind="decode", m=1, n=18944, k=3584, rank=16, adapters=8, none=0.0),
        # a full decode batch, nearly every request with an adapter of its own: the down projection
        dict(name="decode 16 rows", kind="decode", m=16, n=3584, k=18944, rank=32, adapters=16, none=0.1),
        # prompts of several requests in one ragged batch, beside the FP4 product
        dict(name="apply ragged prompts", kind="apply", m=1111, n=11008, k=4096, rank=64, adapters=6, none=0.1, runs=9,
             base=True),
        # a training batch's forward (batch 4 x sequence 2048), one adapter
        dict(name="apply training batch", kind="apply", m=8192, n=4096, k=4096, rank=16, adapters=1, none=0.0, runs=1,
             base=True),
        # a small layer's gradients for a short batch in the parameters' own type: launches count
        dict(name="backward short batch", kind="backward", m=130, n=264, k=520, rank=8, adapters=3, none=0.1, runs=5,
             grad="bf16", base=False),
        # a training batch's gradients at the widest layer, two tasks' adapters, binary32 gradients
        dict(name="backward training batch", kind="backward", m=8192, n=11008, k=4096, rank=16, adapters=2, none=0.02,
             runs=4, grad="f32", base=True),
        # one token of one request with its alternatives
        dict(name="logprobs 1 row", kind="logprobs", rows=1, vocab=128000, dtype="bf16", top=20, temperature=0.7,
             masked=0.0),
        # a decode batch in binary32 with a grammar's mask, an odd vocabulary
        dict(name="logprobs masked batch", kind="logprobs", rows=61, vocab=50257, dtype="f32", top=8, temperature=1.0,
             masked=0.6),
        # the policy loss of a training batch
        dict(name="policy training batch", kind="policy", rows=8192, vocab=32000, dtype="bf16", top=0, temperature=1.0,
             masked=0.0),
        # the residual stream of one decode batch
        dict(name="norm 16 rows", kind="norm", rows=16, cols=3584, x="bf16", res="bf16", post=True, gate=False,
             weight="bf16"),
        # a ragged batch at an odd width in binary32, with a gate for each token
        dict(name="norm odd width", kind="norm_step", rows=1001, cols=1027, x="f32", res="f32", post=True, gate=True,
             weight="f32"),
        # a training batch over a binary32 residual stream
        dict(name="norm training batch", kind="norm_step", rows=8192, cols=4096, x="bf16", res="f32", post=True,
             gate=True, weight="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "apply", "apply", "backward", "backward", "logprobs", "logprobs", "policy",
                       "norm", "norm_step"])
    if kind == "decode":
        return dict(kind=kind, m=rng.randint(1, 16), n=_log(rng, 32, 18944), k=256 * _log(rng, 1, 74),
                    rank=8 * _log(rng, 1, 16), adapters=_log(rng, 1, 32), none=rng.choice([0.0, 0.2]))
    if kind in ("apply", "backward"):
        c = dict(kind=kind, m=_log(rng, 1, 8192), n=8 * _log(rng, 4, 1376), k=8 * _log(rng, 4, 512),
                 rank=8 * _log(rng, 1, 16), adapters=_log(rng, 1, 8), none=rng.choice([0.0, 0.2]),
                 runs=_log(rng, 1, 40), base=rng.random() < 0.7)
        if c["m"] > 2048:
            c["rank"] = min(c["rank"], 16)
        if kind == "backward":
            c["grad"] = rng.choice(["bf16", "f32"])
        return c
    if kind in ("logprobs", "policy"):
        vocab = _log(rng, 100, 128000)
        return dict(kind=kind, rows=min(_log(rng, 1, 8192), 8192 * 30000 // vocab), vocab=vocab,
                    dtype=rng.choice(["bf16", "f32"]), top=rng.choice([0, 1, 5, 20]) if kind == "logprobs" else 0,
                    temperature=rng.choice([1.0, 0.7, 1.3]), masked=rng.choice([0.0, 0.5]))
    return dict(kind=kind, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 4096), x=rng.choice(["bf16", "f32"]),
                res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.8, gate=rng.random() < 0.5,
                weight=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sd=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * sd).to(dtype)


def _fp4_weight(g, n, k):
    """Seeded N(0, 0.02) weights as E2M1 codes with an E4M3 scale for each 16
    elements of a row and a tensor scale: codes [n, k/2] (the even element in
    the low nibble), scale codes [n, k/16], {tensor scale, maximum}."""
    w = _normal(g, (n, k // 16, 16), 0.02)
    top = w.abs().amax()
    ts = top / (6.0 * 448.0)
    sc = (w.abs().amax(-1) / (6.0 * ts)).to(torch.float8_e4m3fn)
    v = w / (sc.float() * ts).clamp_min(1e-30)[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(v.abs(), mids) + 8 * (v < 0)
    code = code.to(torch.uint8).view(n, k // 2, 2)
    return dict(codes=code[..., 0] | (code[..., 1] << 4), scales=sc.view(torch.uint8), ts=torch.stack([ts, top]))


def _runs(g, m, runs, adapters, none):
    """An adapter for each row: contiguous requests of unequal lengths, some without an adapter (-1)."""
    cuts = torch.rand(max(0, runs - 1), generator=g, device="cuda").mul(m).long().sort().values
    run = torch.bucketize(torch.arange(m, device="cuda"), cuts, right=True)
    pick = torch.randint(0, adapters, (runs,), generator=g, device="cuda")
    pick = torch.where(torch.rand(runs, generator=g, device="cuda") < none, -1, pick)
    return pick[run].to(torch.int32)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case)
    if c["kind"] in ("decode", "apply", "backward"):
        m, n, k, r, la = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
        s["x"] = _normal(g, (m, k), 1.0, torch.bfloat16)
        s["a"] = _normal(g, (la, r, k), k ** -0.5, torch.bfloat16)
        s["b"] = _normal(g, (la, n, r), 0.02, torch.bfloat16)
        s["scale"] = torch.rand(la, generator=g, device="cuda") + 1.0
        if c["kind"] == "decode":
            s["w"] = _fp4_weight(g, n, k)
            pick = torch.randperm(max(m, la), generator=g, device="cuda")[:m] % la
            s["slots"] = torch.where(torch.rand(m, generator=g, device="cuda") < c["none"], -1, pick).to(torch.int32)
        else:
            s["slots"] = _runs(g, m, c["runs"], la, c["none"])
        if c["kind"] == "apply":
            s["base"] = _normal(g, (m, n), 1.0, torch.bfloat16) if c["base"] else None
        if c["kind"] == "backward":
            s["dy"] = _normal(g, (m, n), 1e-2, torch.bfloat16)
            s["dx_base"] = _normal(g, (m, k), 1e-2, torch.bfloat16) if c["base"] else None
            s["t"] = _adapter_rows(s["x"], s["a"], s["slots"]).sum(1)
    elif c["kind"] in ("logprobs", "policy"):
        n, v = c["rows"], c["vocab"]
        z = _normal(g, (n, v), 2.5)
        z[torch.arange(n, device="cuda"), torch.randint(0, v, (n,), generator=g, device="cuda")] += 9.0
        tok = torch.randint(0, v, (n,), generator=g, device="cuda")
        if c["masked"]:
            out = torch.rand((n, v), generator=g, device="cuda") < c["masked"]
            out[torch.arange(n, device="cuda"), tok] = False
            z = z.masked_fill(out, float("-inf"))
        s["logits"] = z.to(_DT[c["dtype"]])
        s["tokens"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.05, -100, tok) if n > 1 else tok
        if c["kind"] == "policy":
            s["g_logprob"] = _normal(g, (n,), 1.0 / n)
            s["g_entropy"] = torch.full((n,), -0.01 / n, device="cuda")
    else:
        m, w = c["rows"], c["cols"]
        s["x"] = _normal(g, (m, w), 0.7, _DT[c["x"]])
        s["r"] = _normal(g, (m, w), 2.0, _DT[c["res"]])
        s["w_pre"] = (1.0 + _normal(g, (w,), 0.1)).to(_DT[c["weight"]])
        s["w_post"] = (0.5 + _normal(g, (w,), 0.1)).to(_DT[c["weight"]]) if c["post"] else None
        s["gate"] = torch.rand(m, generator=g, device="cuda") if c["gate"] else None
        s["alpha"], s["eps"] = 0.75, 1e-6
        if c["kind"] == "norm_step":
            s["dn"] = _normal(g, (m, w), 1e-2, _DT[c["x"]])
            s["dh"] = _normal(g, (m, w), 1e-2, _DT[c["res"]])
    return s


# ---------------------------------------------------------------------------
# plain forms, binary32
def _weight(w):
    lut = torch.tensor([*_E2M1, *(-v for v in _E2M1)], device="cuda")
    c = w["codes"].long()
    e = lut[torch.stack([c & 15, c >> 4], -1)].view(c.shape[0], -1, 16)
    return (e * (w["scales"].view(torch.float8_e4m3fn).float() * w["ts"][0])[..., None]).flatten(1)


def _adapter_rows(x, a, slots):
    """[rows, adapters, rank]: x A_a^T in the place of each row's adapter, zero in the others."""
    la, r, k = a.shape
    t = (x.float() @ a.float().view(la * r, k).t()).view(-1, la, r)
    return torch.where((slots[:, None] == torch.arange(la, device="cuda"))[..., None], t, 0.0)


def _columns(b):
    """B [adapters, n, rank] as one [adapters * rank, n] matrix."""
    return b.float().permute(0, 2, 1).reshape(-1, b.shape[1])


def _delta(s):
    t = _adapter_rows(s["x"], s["a"], s["slots"])
    return (t * s["scale"][:, None]).flatten(1) @ _columns(s["b"]), t.sum(1)


def _plain_adapters(s):
    if s["kind"] == "decode":
        return ((s["x"].float() @ _weight(s["w"]).t()) + _delta(s)[0]).bfloat16()
    if s["kind"] == "apply":
        d, t = _delta(s)
        return dict(y=(d if s["base"] is None else s["base"].float() + d).bfloat16(), t=t)
    (la, r, k), n = s["a"].shape, s["b"].shape[1]
    hot = (s["slots"][:, None] == torch.arange(la, device="cuda")).float()[..., None] * s["scale"][:, None]
    dy = s["dy"].float()
    dt = ((dy @ _columns(s["b"]).t()).view(-1, la, r) * hot).flatten(1)
    tt = (s["t"][:, None, :] * hot).flatten(1)
    dx = dt @ s["a"].float().view(la * r, k)
    dx = dx if s["dx_base"] is None else s["dx_base"].float() + dx
    da = (dt.t() @ s["x"].float()).view(la, r, k)
    db = (tt.t() @ dy).view(la, r, n).permute(0, 2, 1)
    return dict(dx=dx.bfloat16(), da=da.to(_DT[s["grad"]]), db=db.to(_DT[s["grad"]]).contiguous())


def _plain_logprobs(s):
    z, v = s["logits"].float(), s["vocab"]
    given = (s["tokens"] >= 0) & (s["tokens"] < v)
    top = z.amax(-1, keepdim=True)
    d = (z - top) / s["temperature"]
    e = d.exp()
    total = e.sum(-1, keepdim=True)
    lp = d - total.log()
    p = e / total
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    hit = lp.gather(1, s["tokens"].clamp(0, v - 1)[:, None])[:, 0]
    out = dict(logprob=torch.where(given, hit, 0.0), entropy=ent)
    if s["top"]:
        ids = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :s["top"]]
        out.update(top_ids=ids.to(torch.int32), top_logprobs=lp.gather(1, ids))
    if s["kind"] == "policy":
        gl = torch.where(given, s["g_logprob"], 0.0)[:, None]
        one = (torch.arange(v, device="cuda") == s["tokens"][:, None]).float()
        ge = s["g_entropy"][:, None]
        dz = gl * (one - p) - ge * torch.where(p > 0, p * (lp + ent[:, None]), 0.0)
        out["dlogits"] = (dz / s["temperature"]).to(s["logits"].dtype)
    return out


def _plain_norm(s):
    x, r, w = s["x"].float(), s["r"].float(), s["cols"]
    w2 = s["w_pre"].float()
    r1 = (x.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
    w1 = s["w_post"].float() if s["post"] else None
    u = x * r1 * w1 if s["post"] else x
    gate = s["gate"][:, None] if s["gate"] is not None else 1.0
    h = s["alpha"] * r + gate * u
    r2 = (h.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
    out = dict(h=h.to(s["r"].dtype), n=(h * r2 * w2).to(s["x"].dtype))
    if s["kind"] == "norm":
        return out
    dn, dh = s["dn"].float(), s["dh"].float()
    q = dn * w2
    dh = dh + r2 * q - h * r2.pow(3) * (q * h).sum(-1, keepdim=True) / w
    out["dw_pre"] = (dn * h * r2).sum(0)
    out["dr"] = (s["alpha"] * dh).to(s["r"].dtype)
    if s["gate"] is not None:
        out["dgate"] = (dh * u).sum(-1)
    du = gate * dh
    if s["post"]:
        out["dw_post"] = (du * x * r1).sum(0)
        q = du * w1
        du = r1 * q - x * r1.pow(3) * (q * x).sum(-1, keepdim=True) / w
    out["dx"] = du.to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------
# the package's entry points
def _own(s):
    import fp4_block_scaled_quantize_amd as fq
    kind = s["kind"]
    if kind in ("decode", "apply", "backward"):
        bank = fq.LoraBank(s["a"], s["b"], s["scale"])
        if kind == "decode":
            w = s["w"]
            q = fq.QTensor(w["codes"], w["scales"], w["ts"], s["n"], s["k"], 16, "e4m3")
            return fq.fp4_wo_gemm_lora(s["x"], q, bank, s["slots"])
        if kind == "apply":
            y, t = fq.fp4_lora_apply(s["x"], bank, s["slots"], base=s["base"])
            return dict(y=y, t=t)
        dx, da, db = fq.fp4_lora_backward(s["dy"], s["x"], s["t"], bank, s["slots"], dx_base=s["dx_base"],
                                          grad_dtype=_DT[s["grad"]])
        return dict(dx=dx, da=da, db=db)
    if kind in ("logprobs", "policy"):
        f = fq.fp4_token_logprobs(s["logits"], s["tokens"], temperature=s["temperature"], top=s["top"])
        out = dict(logprob=f.logprob, entropy=f.entropy)
        if s["top"]:
            out.update(top_ids=f.top_ids, top_logprobs=f.top_logprobs)
        if kind == "policy":
            out["dlogits"] = fq.fp4_token_logprobs_backward(s["logits"], s["tokens"], f, s["g_logprob"],
                                                            s["g_entropy"], temperature=s["temperature"])
        return out
    h, n, stats = fq.fp4_residual_norm(s["x"], s["r"], s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                       alpha=s["alpha"], eps=s["eps"])
    out = dict(h=h, n=n)
    if kind == "norm_step":
        d = fq.fp4_residual_norm_backward(s["dn"], s["dh"], s["x"], s["r"], s["w_pre"], stats, w_post=s["w_post"],
                                          gate=s["gate"], alpha=s["alpha"])
        out.update(dx=d.dx, dr=d.dres, dw_pre=d.dw_pre)
        if s["gate"] is not None:
            out["dgate"] = d.dgate
        if s["post"]:
            out["dw_post"] = d.dw_post
    return out


def run(state):
    if own:
        return _own(state)
    if state["kind"] in ("decode", "apply", "backward"):
        return _plain_adapters(state)
    return _plain_logprobs(state) if state["kind"] in ("logprobs", "policy") else _plain_norm(state)


# ---------------------------------------------------------------------------
# binary64, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["kind"] in ("decode", "apply", "backward"):
        x, la = s["x"].to(f), case["adapters"]
        t = torch.zeros(case["m"], case["rank"], dtype=f, device="cuda")
        d = torch.zeros(case["m"], case["n"], dtype=f, device="cuda")
        rows = [(s["slots"] == i).nonzero()[:, 0] for i in range(la)]
        a, b, sc = s["a"].to(f), s["b"].to(f), s["scale"].to(f)
        if case["kind"] != "backward":
            for i, at in enumerate(rows):
                t[at] = x[at] @ a[i].t()
                d[at] = sc[i] * (t[at] @ b[i].t().contiguous())
            if case["kind"] == "apply":
                return dict(y=d if s["base"] is None else s["base"].to(f) + d, t=t)
            lo, hi = s["w"]["codes"] & 15, s["w"]["codes"] >> 4
            c = torch.stack([lo, hi], -1).flatten(1).to(torch.int32)
            mag = c & 7
            e = torch.exp2((mag >> 1).to(f) - 1.0)
            val = torch.where(mag < 2, 0.5 * mag.to(f), (1.0 + 0.5 * (mag & 1).to(f)) * e)
            val = torch.where(c >= 8, -val, val)
            wt = s["w"]["scales"].view(torch.float8_e4m3fn).to(f) * s["w"]["ts"][0].to(f)
            return x @ (val * wt.repeat_interleave(16, 1)).t() + d
        dy, tt = s["dy"].to(f), s["t"].to(f)
        dx = torch.zeros_like(x) if s["dx_base"] is None else s["dx_base"].to(f)
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for i, at in enumerate(rows):
            dt = sc[i] * (dy[at] @ b[i])
            dx[at] += dt @ a[i]
            da[i] = dt.t() @ x[at]
            db[i] = sc[i] * (dy[at].t() @ tt[at])
        return dict(dx=dx, da=da, db=db)
    if case["kind"] in ("logprobs", "policy"):
        z = s["logits"].to(f) / case["temperature"]
        lse = torch.logsumexp(z, -1)
        lp = z - lse[:, None]
        p = lp.exp()
        ent = lse - (p * z.masked_fill(p == 0, 0.0)).sum(-1)
        ok = s["tokens"] >= 0
        at = s["tokens"].clamp_min(0)
        out = dict(logprob=torch.where(ok, lp[torch.arange(len(at), device="cuda"), at], 0.0), entropy=ent)
        if case["top"]:
            v, i = torch.sort(lp, dim=-1, descending=True, stable=True)
            out.update(top_ids=i[:, :case["top"]].to(torch.int32), top_logprobs=v[:, :case["top"]])
        if case["kind"] == "policy":
            gl = torch.where(ok, s["g_logprob"].to(f), 0.0)
            dz = -p * (gl[:, None] + s["g_entropy"].to(f)[:, None] * (lp.masked_fill(p == 0, 0.0) + ent[:, None]))
            dz[torch.arange(len(at), device="cuda"), at] += gl
            out["dlogits"] = dz / case["temperature"]
        return out
    x, r = s["x"].to(f), s["r"].to(f)
    w1 = s["w_post"].to(f) if case["post"] else torch.ones(case["cols"], dtype=f, device="cuda")
    w2 = s["w_pre"].to(f)
    gate = s["gate"].to(f) if case["gate"] else torch.ones(case["rows"], dtype=f, device="cuda")
    leaves = [v.requires_grad_(case["kind"] == "norm_step") for v in (x, r, w1, w2, gate)]
    u = x / (x.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w1 if case["post"] else x
    h = s["alpha"] * r + gate[:, None] * u
    n = h / (h.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w2
    out = dict(h=h.detach(), n=n.detach())
    if case["kind"] == "norm_step":
        names = ("dx", "dr", "dw_post", "dw_pre", "dgate")
        got = torch.autograd.grad((h, n), leaves, (s["dh"].to(f), s["dn"].to(f)), allow_unused=True)
        out.update({k: v for k, v in zip(names, got)
                    if (k != "dgate" or case["gate"]) and (k != "dw_post" or case["post"])})
    return out


# ---------------------------------------------------------------------------
def work(case):
    c, sz = case, {"bf16": 2, "f32": 4}
    if c["kind"] in ("decode", "apply", "backward"):
        m, n, k, r = c["m"], c["n"], c["k"], c["rank"]
        used = min(c["adapters"], m if c["kind"] == "decode" else c["runs"])
        bank = 2 * used * r * (n + k)
        if c["kind"] == "decode":
            return {"bytes": n * k * 9 / 16 + bank + 2 * m * (n + k), "flops": 2.0 * m * n * k + 2.0 * m * r * (n + k)}
        if c["kind"] == "apply":
            return {"bytes": bank + 2 * m * k + 2 * m * n * (2 if c["base"] else 1) + 4 * m * r,
                    "flops": 2.0 * m * r * (n + k)}
        grads = c["adapters"] * r * (n + k) * sz[c["grad"]]
        return {"bytes": bank + grads + 2 * m * n + 2 * m * k * (3 if c["base"] else 2) + 4 * m * r,
                "flops": 4.0 * m * r * (n + k)}
    if c["kind"] in ("logprobs", "policy"):
        n, v, e = c["rows"], c["vocab"], sz[c["dtype"]]
        step = c["kind"] == "policy"
        # the backward pass reads the logits again: a row's sums are known only after its last element
        return {"bytes": n * v * e * (3 if step else 1) + n * (24 + 8 * c["top"]),
                "flops": n * v * (16.0 if step else 8.0)}
    m, w, ex, er = c["rows"], c["cols"], sz[c["x"]], sz[c["res"]]
    fwd = 2 * m * w * (ex + er)
    step = c["kind"] == "norm_step"
    return {"bytes": fwd + (3 * m * w * (ex + er) if step else 0) + 2 * w * sz[c["weight"]],
            "flops": m * w * (30.0 if step else 10.0)}
