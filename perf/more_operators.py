"""Cases of the fused product epilogues, the mixture-of-experts layer and the distillation loss.

Every case is one call, or the calls that go together, as a program that
serves a model with FP4 weights, or trains one from a full-precision teacher,
makes them.  `run` computes it from elementary torch operations in binary32
(rounded once, at the end) or, where `own` is set, through the package's
entry points; `exact` computes it in binary64.

Kinds of a case:
  wo          y = residual + mul act(x W^T + bias) for at most 16 rows, W quantized
  product     the same of two quantized operands; in training also the rounded x W^T + bias that the backward pass reads
  step        the gradients of the epilogue: of x W^T + bias, of bias and of mul
  moe         the router's choice among the experts and the layer y = residual + sum_k w_k act(x G_k^T) (x U_k^T) D_k^T
  distill     the loss against a teacher's top log probabilities and the gradient of the student's logits
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# element grid, block, scale encoding, policy of the tensor maximum
_FORMATS = {"nvfp4": ("e2m1", 16, "e4m3", "current"), "mxfp4": ("e2m1", 32, "e8m0", "none"),
            "mxfp8": ("fp8_e4m3", 32, "e8m0", "none")}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one request being generated: an attention projection with its bias, one token
        dict(name="wo 1 row, bias", kind="wo", m=1, n=3584, k=3584, fmt="nvfp4", bias="bf16", act="none", mul=False,
             residual=False),
        # a full decode batch: the gate projection, multiplied into the up projection's output
        dict(name="wo 16 rows, gated", kind="wo", m=16, n=18944, k=3584, fmt="nvfp4", bias="", act="silu", mul=True,
             residual=False),
        # the small configuration as one layer
        dict(name="product small", kind="product", m=64, n=256, k=256, fmt="nvfp4", bias="f32", act="gelu", mul=False,
             residual=True, pre=False),
        # prompts of several requests in one ragged batch: the down projection into the residual stream
        dict(name="product ragged prompts", kind="product", m=1111, n=4096, k=11008, fmt="nvfp4", bias="", act="none",
             mul=False, residual=True, pre=False),
        # a training batch's gate projection (batch 4 x sequence 2048)
        dict(name="product training batch", kind="product", m=8192, n=11008, k=4096, fmt="mxfp4", bias="bf16",
             act="silu", mul=True, residual=False, pre=True),
        # a ragged short batch's backward pass: launches count
        dict(name="step short batch", kind="step", m=130, n=1027, act="gelu", mul=False, bias=True),
        # the training batch's backward pass
        dict(name="step training batch", kind="step", m=8192, n=11008, act="silu", mul=True, bias=True),
        # one token of one request through many narrow experts
        dict(name="moe 1 token", kind="moe", m=1, hidden=2048, ffn=768, experts=128, top=8, fmt="nvfp4", act="silu",
             score="softmax", residual=True),
        # a few requests through few wide experts
        dict(name="moe 3 tokens", kind="moe", m=3, hidden=4096, ffn=11008, experts=8, top=2, fmt="mxfp4", act="silu",
             score="softmax", residual=False),
        # a full decode batch through many experts, scored one by one with a balancing bias
        dict(name="moe 16 tokens", kind="moe", m=16, hidden=4096, ffn=1536, experts=64, top=6, fmt="nvfp4", act="silu",
             score="sigmoid", residual=True),
        # a short sequence of a student with an odd vocabulary, only the listed tokens counted
        dict(name="distill short sequence", kind="distill", rows=61, vocab=50257, dtype="f32", top=8, temperature=1.0,
             rest="renormalize", padded=0.05),
        # a training batch
        dict(name="distill training batch", kind="distill", rows=8192, vocab=32000, dtype="bf16", top=32,
             temperature=2.0, rest="bucket", padded=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["wo", "wo", "product", "product", "step", "moe", "moe", "moe", "distill", "distill"])
    c = dict(kind=kind)
    if kind in ("wo", "product"):
        c.update(fmt=rng.choice(list(_FORMATS)), bias=rng.choice(["", "bf16", "f32"]), act=rng.choice(_ACTS),
                 mul=rng.random() < 0.5, residual=rng.random() < 0.5)
        if kind == "wo":
            c.update(m=rng.randint(1, 16), n=_log(rng, 32, 18944), k=256 * _log(rng, 1, 74))
        else:
            c.update(m=_log(rng, 1, 8192), n=_log(rng, 32, 11008), k=128 * _log(rng, 1, 32), pre=rng.random() < 0.5)
    elif kind == "step":
        c.update(m=_log(rng, 1, 8192), n=_log(rng, 32, 11008), act=rng.choice(_ACTS[1:]), mul=rng.random() < 0.5,
                 bias=rng.random() < 0.7)
    elif kind == "moe":
        hidden, ffn = 256 * _log(rng, 1, 16), 256 * _log(rng, 1, 43)
        experts = _log(rng, 2, min(128, max(2, 64 * 4096 * 1536 // (hidden * ffn))))
        c.update(m=rng.randint(1, 16), hidden=hidden, ffn=ffn, experts=experts, top=rng.randint(1, min(8, experts)),
                 fmt=rng.choice(list(_FORMATS)), act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                 score=rng.choice(["softmax", "sigmoid"]), residual=rng.random() < 0.5)
    else:
        vocab = _log(rng, 300, 128000)
        c.update(rows=min(_log(rng, 1, 8192), 8192 * 30000 // vocab), vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                 top=_log(rng, 1, 100), temperature=rng.choice([1.0, 0.7, 2.0]),
                 rest=rng.choice(["bucket", "renormalize"]), padded=rng.choice([0.0, 0.3]))
    return c


# ---------------------------------------------------------------------------
# inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sd=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * sd).to(dtype)


def _quantized(g, rows, cols, sd, fmt):
    """Seeded N(0, sd) values as codes, scale codes for each block of a row, and {tensor scale, maximum}."""
    elem, block, enc, _ = _FORMATS[fmt]
    w = _normal(g, (rows, cols // block, block), sd)
    amax = w.abs().amax(-1)
    top = amax.amax()
    big = 6.0 if elem == "e2m1" else 448.0
    if enc == "e4m3":
        ts = top / (6.0 * 448.0)
        sc = (amax / (6.0 * ts)).to(torch.float8_e4m3fn)
        step, sc = sc.float() * ts, sc.view(torch.uint8)
    else:
        ts = torch.ones((), device="cuda")
        e = torch.floor(torch.log2(amax.clamp_min(1e-30))) - (2.0 if elem == "e2m1" else 8.0)
        step, sc = torch.exp2(e), (e + 127.0).to(torch.uint8)
    v = (w / step.clamp_min(1e-30)[..., None]).clamp(-big, big)
    if elem == "e2m1":
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        code = torch.bucketize(v.abs(), mids, out_int32=True) + 8 * (v < 0)
        code = code.to(torch.uint8).view(rows, cols // 2, 2)
        code = code[..., 0] | (code[..., 1] << 4)
    else:
        code = v.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, cols)
    return dict(codes=code, scales=sc, ts=torch.stack([ts, top]), rows=rows, cols=cols, fmt=fmt)


def _experts(g, experts, rows, cols, sd, fmt):
    """Experts' matrices below one another, each quantized on its own: its tensor scale is one of `each`."""
    parts = [_quantized(g, rows, cols, sd, fmt) for _ in range(experts)]
    return dict(codes=torch.cat([p["codes"] for p in parts]), scales=torch.cat([p["scales"] for p in parts]),
                ts=torch.ones(2, device="cuda"), rows=experts * rows, cols=cols, fmt=fmt,
                each=torch.stack([p["ts"][0] for p in parts]))


def prepare(case, seed):
    g, c = _gen(seed), case
    s = dict(case)
    if c["kind"] in ("wo", "product"):
        m, n, k = c["m"], c["n"], c["k"]
        s["w"] = _quantized(g, n, k, 0.02, c["fmt"])
        s["x"] = _normal(g, (m, k), 1.0, torch.bfloat16) if c["kind"] == "wo" else _quantized(g, m, k, 1.0, c["fmt"])
        s["b"] = _normal(g, (n,), 0.5, _DT[c["bias"]]) if c["bias"] else None
        s["mu"] = _normal(g, (m, n), 1.0, torch.bfloat16) if c["mul"] else None
        s["r"] = _normal(g, (m, n), 2.0, torch.bfloat16) if c["residual"] else None
    elif c["kind"] == "step":
        m, n = c["m"], c["n"]
        s["pre"] = _normal(g, (m, n), 1.5, torch.bfloat16)
        s["dy"] = _normal(g, (m, n), 1e-2, torch.bfloat16)
        s["mu"] = _normal(g, (m, n), 1.0, torch.bfloat16) if c["mul"] else None
    elif c["kind"] == "moe":
        m, h, f, e = c["m"], c["hidden"], c["ffn"], c["experts"]
        s["up"] = _experts(g, e, 2 * f, h, 0.02, c["fmt"])
        s["down"] = _experts(g, e, h, f, 0.02, c["fmt"])
        s["x"] = _normal(g, (m, h), 1.0, torch.bfloat16)
        s["logits"] = _normal(g, (m, e), 1.5)
        s["bias"] = _normal(g, (e,), 0.1) if c["score"] == "sigmoid" else None
        s["r"] = _normal(g, (m, h), 2.0, torch.bfloat16) if c["residual"] else None
    else:
        n, v, k = c["rows"], c["vocab"], c["top"]
        z = _normal(g, (n, v), 2.5)
        z[torch.arange(n, device="cuda"), torch.randint(0, v, (n,), generator=g, device="cuda")] += 9.0
        s["logits"] = (z + _normal(g, (n, v), 0.5)).to(_DT[c["dtype"]])
        top = torch.topk(z, k, dim=-1)
        lse = torch.logsumexp(z / c["temperature"], -1, keepdim=True)
        s["lp"] = top.values / c["temperature"] - lse
        pad = torch.rand(n, generator=g, device="cuda") < c["padded"]
        s["ids"] = torch.where(pad[:, None], -1, top.indices).to(torch.int32)
        s["g"] = torch.rand(n, generator=g, device="cuda") / n
    return s


# ---------------------------------------------------------------------------
# plain forms, binary32
def _values(w, lo=0, hi=None):
    """Rows lo .. hi of a quantized matrix."""
    elem, block, enc, _ = _FORMATS[w["fmt"]]
    c, sc = w["codes"][lo:hi], w["scales"][lo:hi]
    if elem == "e2m1":
        lut = torch.tensor([*_E2M1, *(-v for v in _E2M1)], device="cuda")
        e = lut[torch.stack([c & 15, c >> 4], -1).int()].flatten(1)
    else:
        e = c.view(torch.float8_e4m3fn).float()
    step = sc.view(torch.float8_e4m3fn).float() if enc == "e4m3" else torch.exp2(sc.float() - 127.0)
    return (e.view(e.shape[0], -1, block) * (step * w["ts"][0])[..., None]).flatten(1)


def _act(v, act):
    if act == "relu":
        return v.clamp_min(0.0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v * v * v))
    return v


def _slope(v, act):
    if act == "relu":
        return (v > 0).float()
    if act == "silu":
        return torch.sigmoid(v) * (1.0 + v * torch.sigmoid(-v))
    if act == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(8.0 / math.pi)
        u = c * (v + 0.044715 * v * v * v)
        return torch.sigmoid(u) * (1.0 + v * torch.sigmoid(-u) * c * (1.0 + 3 * 0.044715 * v * v))
    return torch.ones_like(v)


def _plain_product(s):
    x = s["x"].float() if s["kind"] == "wo" else _values(s["x"])
    v = x @ _values(s["w"]).t()
    if s["b"] is not None:
        v = v + s["b"].float()
    y = _act(v, s["act"])
    if s["mu"] is not None:
        y = s["mu"].float() * y
    if s["r"] is not None:
        y = s["r"].float() + y
    out = dict(y=y.bfloat16())
    if s["kind"] == "product" and s["pre"]:
        out["pre"] = v.bfloat16()
    return out


def _plain_step(s):
    dy, v = s["dy"].float(), s["pre"].float()
    du = dy * s["mu"].float() if s["mul"] else dy
    dv = du * _slope(v, s["act"])
    out = dict(dpre=dv.bfloat16())
    if s["mul"]:
        out["dmul"] = (dy * _act(v, s["act"])).bfloat16()
    if s["bias"]:
        out["dbias"] = dv.sum(0)
    return out


def _plain_moe(s):
    f, h, e = s["ffn"], s["hidden"], s["experts"]
    z = s["logits"].double()                # a choice goes by the scores' order: next to each other in 64 bits
    score = torch.softmax(z, -1) if s["score"] == "softmax" else torch.sigmoid(z)
    by = score if s["bias"] is None else score + s["bias"].double()
    ids = torch.sort(by, dim=-1, descending=True, stable=True).indices[:, :s["top"]]
    p = score.gather(1, ids)
    p = (p / p.sum(-1, keepdim=True)).float()
    x, y = s["x"].float(), torch.zeros_like(s["x"], dtype=torch.float32)
    for i in range(e):
        mine = ids == i
        gu = (x @ _values(s["up"], 2 * f * i, 2 * f * (i + 1)).t()) * s["up"]["each"][i]
        a = _act(gu[:, :f], s["act"]) * gu[:, f:]
        o = (a @ _values(s["down"], h * i, h * (i + 1)).t()) * s["down"]["each"][i]
        w = torch.where(mine, p, 0.0).sum(-1, keepdim=True)
        y = torch.where(mine.any(-1, keepdim=True), y + w * o, y)
    y = y if s["r"] is None else s["r"].float() + y
    return dict(ids=ids.to(torch.int32), weights=p, y=y.bfloat16())


def _plain_distill(s):
    # a loss is a small difference of large terms: a row's sums and what they give in 64 bits
    z, c = s["logits"].float(), 1.0 / s["temperature"]
    has = s["ids"] >= 0
    at = s["ids"].long().clamp_min(0)
    t = s["lp"].double()
    p = torch.where(has, t.exp(), 0.0)
    mass = p.sum(-1, keepdim=True)
    if s["rest"] == "renormalize":
        t = t - mass.log()
        p = torch.where(has, p / mass, 0.0)
    top = z.amax(-1, keepdim=True)
    e = ((z - top) * c).exp()
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    lq = (z.gather(1, at).double() - top.double()) * c - total.log()
    loss = torch.where(has, p * (t - lq), 0.0).sum(-1)
    q = e / total.float()
    listed_mass = torch.zeros_like(q).scatter_add(1, at, p.float())
    grad = torch.where(mass > 0, q - listed_mass, 0.0)
    if s["rest"] == "bucket":
        hit = torch.zeros_like(q).scatter_add(1, at, has.float()) > 0
        left = (1.0 - mass).clamp_min(0.0)
        rest = torch.where(hit, 0.0, e).sum(-1, keepdim=True, dtype=torch.float64) / total
        some = (left > 0) & (rest > 0) & (mass > 0)
        loss = loss + torch.where(some, left * (left.log() - rest.log()), 0.0)[:, 0]
        ratio = torch.where(some, left / rest, 0.0)
        # a row without a tail term: the listed probabilities alone
        full = torch.where(some, 1.0, mass)
        grad = torch.where(hit, full.float() * q - listed_mass, q * (full - ratio).float())
        grad = torch.where(mass > 0, grad, 0.0)
    dz = s["g"][:, None] * c * grad
    return dict(loss=torch.where(mass[:, 0] > 0, loss, 0.0).float(), dlogits=dz.to(s["logits"].dtype))


# ---------------------------------------------------------------------------
# the package's entry points
def _tensor(fq, w):
    elem, block, enc, policy = _FORMATS[w["fmt"]]
    return fq.QTensor(w["codes"], w["scales"], w["ts"], w["rows"], w["cols"], block, enc, amax=policy, element=elem)


def _own(s):
    import fp4_block_scaled_quantize_amd as fq
    kind = s["kind"]
    if kind == "wo":
        return dict(y=fq.fp4_wo_gemm_epilogue(s["x"], _tensor(fq, s["w"]), bias=s["b"], act=s["act"], mul=s["mu"],
                                              residual=s["r"]))
    if kind == "product":
        y, pre = fq.fp4_gemm_epilogue(_tensor(fq, s["x"]), _tensor(fq, s["w"]), bias=s["b"], act=s["act"], mul=s["mu"],
                                      residual=s["r"], save_pre=s["pre"])
        return dict(y=y, pre=pre) if s["pre"] else dict(y=y)
    if kind == "step":
        d = fq.fp4_epilogue_backward(s["dy"], s["pre"], act=s["act"], mul=s["mu"], bias=s["bias"])
        out = dict(dpre=d.dpre)
        if s["mul"]:
            out["dmul"] = d.dmul
        if s["bias"]:
            out["dbias"] = d.dbias
        return out
    if kind == "moe":
        ids, weights = fq.fp4_moe_route(s["logits"], s["top"], score=s["score"], bias=s["bias"])
        bank = fq.MoeBank(_tensor(fq, s["up"]), _tensor(fq, s["down"]), s["experts"], up_scale=s["up"]["each"],
                          down_scale=s["down"]["each"])
        return dict(ids=ids, weights=weights, y=fq.fp4_moe(s["x"], bank, ids, weights, act=s["act"], residual=s["r"]))
    f = fq.fp4_distill_loss(s["logits"], s["ids"], s["lp"], temperature=s["temperature"], rest=s["rest"])
    dz = fq.fp4_distill_loss_backward(s["logits"], s["ids"], s["lp"], f, s["g"], temperature=s["temperature"],
                                      rest=s["rest"])
    return dict(loss=f.loss, dlogits=dz)


def run(state):
    if own:
        return _own(state)
    return {"wo": _plain_product, "product": _plain_product, "step": _plain_step, "moe": _plain_moe,
            "distill": _plain_distill}[state["kind"]](state)


# ---------------------------------------------------------------------------
# binary64, from the definitions
def _exact_matrix(w, lo=0, hi=None):
    elem, block, enc, _ = _FORMATS[w["fmt"]]
    f = torch.float64
    c = w["codes"][lo:hi].int()
    if elem == "e2m1":
        c = torch.stack([c % 16, c // 16], -1).flatten(1)
        mag = c % 8
        v = torch.where(mag < 2, 0.5 * mag.to(f), (1.0 + 0.5 * (mag % 2).to(f)) * torch.exp2((mag // 2).to(f) - 1.0))
        v = torch.where(c >= 8, -v, v)
    else:
        e, m = (c // 8) % 16, (c % 8).to(f) / 8.0
        v = torch.where(e == 0, m * 2.0 ** -6, (1.0 + m) * torch.exp2(e.to(f) - 7.0))
        v = torch.where(c >= 128, -v, v)
    b = w["scales"][lo:hi].int()
    if enc == "e4m3":
        e, m = (b // 8) % 16, (b % 8).to(f) / 8.0
        sc = torch.where(e == 0, m * 2.0 ** -6, (1.0 + m) * torch.exp2(e.to(f) - 7.0))
    else:
        sc = torch.exp2(b.to(f) - 127.0)
    return v * sc.repeat_interleave(block, 1) * w["ts"][0].to(f)


def _exact_act(v, act):
    if act == "none":
        return v
    if act == "relu":
        return torch.where(v > 0, v, 0.0)
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return v * torch.special.ndtr(v)
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["kind"] in ("wo", "product"):
        x = s["x"].to(f) if case["kind"] == "wo" else _exact_matrix(s["x"])
        v = x @ _exact_matrix(s["w"]).t()
        if case["bias"]:
            v += s["b"].to(f)
        y = _exact_act(v, case["act"])
        y = y * s["mu"].to(f) if case["mul"] else y
        y = y + s["r"].to(f) if case["residual"] else y
        return dict(y=y, pre=v) if case.get("pre") else dict(y=y)
    if case["kind"] == "step":
        v, dy = s["pre"].to(f).requires_grad_(True), s["dy"].to(f)
        u = _exact_act(v, case["act"])
        out = dict(dpre=torch.autograd.grad(u, v, dy * s["mu"].to(f) if case["mul"] else dy)[0])
        if case["mul"]:
            out["dmul"] = dy * u.detach()
        if case["bias"]:
            out["dbias"] = out["dpre"].sum(0)
        return out
    if case["kind"] == "moe":
        z = s["logits"].to(f)
        sc = z.exp() / z.exp().sum(-1, keepdim=True) if case["score"] == "softmax" else 1.0 / (1.0 + (-z).exp())
        by = sc + s["bias"].to(f) if s["bias"] is not None else sc
        ids = torch.argsort(by, dim=-1, descending=True, stable=True)[:, :case["top"]]
        w = torch.take_along_dim(sc, ids, 1)
        w = w / w.sum(-1, keepdim=True)
        x, n, h = s["x"].to(f), case["ffn"], case["hidden"]
        y = torch.zeros_like(x) if s["r"] is None else s["r"].to(f)
        for i in ids.unique().tolist():
            row, col = (ids == i).nonzero(as_tuple=True)
            up = _exact_matrix(s["up"], 2 * n * i, 2 * n * (i + 1)) * s["up"]["each"][i].to(f)
            down = _exact_matrix(s["down"], h * i, h * (i + 1)) * s["down"]["each"][i].to(f)
            a = _exact_act(x[row] @ up[:n].t(), case["act"]) * (x[row] @ up[n:].t())
            y[row] += w[row, col][:, None] * (a @ down.t())
        return dict(ids=ids.to(torch.int32), weights=w, y=y)
    ids, lp, c = s["ids"].long(), s["lp"].to(f), 1.0 / case["temperature"]
    used = ids[:, 0] >= 0
    zz = s["logits"].to(f)
    loss = torch.zeros(case["rows"], dtype=f, device="cuda")
    dz = torch.zeros_like(zz)
    for at in used.nonzero()[:, 0].split(256):
        z = zz[at].requires_grad_(True)
        q = torch.log_softmax(z * c, -1)
        lq, t = torch.take_along_dim(q, ids[at], 1), lp[at]
        mass = t.exp().sum(-1, keepdim=True)
        if case["rest"] == "renormalize":
            each = (t.exp() / mass * (t - mass.log() - lq)).sum(-1)
        else:
            each = (t.exp() * (t - lq)).sum(-1)
            left = (1.0 - mass[:, 0]).clamp_min(0.0)
            rest = torch.logsumexp(q.scatter(1, ids[at], float("-inf")), -1)
            some = (left > 0) & (rest > float("-inf"))
            each = each + torch.where(some, left * (left.clamp_min(1e-300).log() - rest.clamp_min(-1e300)), 0.0)
        loss[at] = each.detach()
        dz[at] = torch.autograd.grad(each, z, s["g"][at].to(f))[0]
    return dict(loss=loss, dlogits=dz)


# ---------------------------------------------------------------------------
def work(case):
    c, sz = case, {"bf16": 2, "f32": 4, "": 0}
    bits = {"nvfp4": 4.5, "mxfp4": 4.25, "mxfp8": 8.25}
    if c["kind"] in ("wo", "product"):
        m, n, k = c["m"], c["n"], c["k"]
        x = 2.0 * m * k if c["kind"] == "wo" else m * k * bits[c["fmt"]] / 8
        outs = 1 + bool(c["mul"]) + bool(c["residual"]) + bool(c.get("pre"))
        return {"bytes": x + n * k * bits[c["fmt"]] / 8 + 2.0 * m * n * outs + n * sz[c["bias"]],
                "flops": 2.0 * m * n * k}
    if c["kind"] == "step":
        m, n = c["m"], c["n"]
        return {"bytes": 2.0 * m * n * (5 if c["mul"] else 3) + 4.0 * n * bool(c["bias"]), "flops": 20.0 * m * n}
    if c["kind"] == "moe":
        m, h, f, e, k = c["m"], c["hidden"], c["ffn"], c["experts"], c["top"]
        # experts that a batch of evenly spread choices meets
        met = e * (1.0 - (1.0 - k / e) ** m)
        return {"bytes": met * 3 * h * f * bits[c["fmt"]] / 8 + 2.0 * m * h * (3 if c["residual"] else 2) + 4.0 * m * e,
                "flops": 6.0 * m * k * h * f}
    n, v, e = c["rows"], c["vocab"], sz[c["dtype"]]
    # a padded row's gradient is written without reading its logits; the backward pass reads the others again: a row's
    # sums are known only after its last element
    return {"bytes": n * v * e * (1.0 + 2.0 * (1.0 - c["padded"])) + n * (8 * c["top"] + 8),
            "flops": n * v * 12.0}
