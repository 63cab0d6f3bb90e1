"""Cases for measuring a drafted decode step's operators, each with a plain form.

Three operators, in the order a step of speculative decoding runs them on its few tokens, and the trainer's side of one:

  moe     the whole mixture-of-experts layer of at most 16 tokens: router, choice, gate/up product, SwiGLU, down product,
          shared expert and combine
  norm    the norms after and before a block: the block's output normalised, gated and scaled, added to the scaled residual
          stream, and that row normalised for the next block; its backward
  verify  drafted tokens checked against the target's probabilities from given random numbers, and the token that follows
          the last accepted one

`own` chooses between the plain forms here (elementary torch operations in 32 bits, in 64 where a choice hangs on them) and
the framework's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- cases

def listed():
    qwen = {"E": 128, "H": 2048, "F": 768, "shared": 0, "k": 8}
    glm = {"E": 256, "H": 6144, "F": 2048, "shared": 2048, "k": 8}
    soft = {"score": "topk", "bias": False, "groups": 1, "topk_groups": 1, "renorm": True, "scale": 1.0}
    scored = {"score": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "renorm": True, "scale": 2.5}
    return [
        # one token through the tiny layer: latency only
        {"name": "moe_tiny_one", "op": "moe", "T": 1, "E": 8, "H": 256, "F": 512, "shared": 0, "k": 2, **soft},
        # one token of one request
        {"name": "moe_qwen_one", "op": "moe", "T": 1, **qwen, **soft},
        # four requests with three drafted tokens each
        {"name": "moe_qwen_drafts", "op": "moe", "T": 16, **qwen, **soft},
        # one token of one request through the layer with a shared expert
        {"name": "moe_glm_one", "op": "moe", "T": 1, **glm, **soft},
        # one request with seven drafted tokens, experts chosen by score and balance bias inside the best groups
        {"name": "moe_glm_drafts", "op": "moe", "T": 8, **glm, **scored},
        # the eight rows of that step between two blocks: latency only
        {"name": "norm_decode", "op": "norm", "T": 8, "H": 6144, "x": "fp32", "res": "bf16", "gate": "none", "next": True,
         "res_scale": 1.0, "branch_scale": 1.0},
        # a prefill step: the layer's fp32 output, a gate per channel
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 6144, "x": "fp32", "res": "bf16", "gate": "channel",
         "next": True, "res_scale": 1.0, "branch_scale": 0.25},
        # the trainer's side of the 2048-wide block, a gate per token and an fp32 residual stream
        {"name": "norm_backward_token", "op": "norm_bwd", "T": 4096, "H": 2048, "x": "fp32", "res": "fp32", "dy": "fp32",
         "gate": "token", "next": True, "res_scale": 0.875, "branch_scale": 1.0},
        # the trainer's side of the prefill step
        {"name": "norm_backward", "op": "norm_bwd", "T": 8192, "H": 6144, "x": "fp32", "res": "bf16", "dy": "bf16",
         "gate": "channel", "next": True, "res_scale": 1.0, "branch_scale": 0.25},
        # the next token of eight requests without drafts, a small vocabulary: latency only
        {"name": "verify_sample_small", "op": "verify", "B": 8, "D": 0, "V": 4096, "logits": "fp32", "draft": "none",
         "ragged": False, "temperature": "one"},
        # four drafted tokens of one request
        {"name": "verify_one", "op": "verify", "B": 1, "D": 4, "V": 151552, "logits": "fp32", "draft": "logits",
         "ragged": False, "temperature": "one"},
        # up to four drafted tokens for each of 64 requests with temperatures of their own, some of them greedy
        {"name": "verify_batch", "op": "verify", "B": 64, "D": 4, "V": 151552, "logits": "fp32", "draft": "logits",
         "ragged": True, "temperature": "each"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    return max(lo, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["moe", "moe", "norm", "norm_bwd", "verify", "verify"])
    if op == "moe":
        groups, per = rng.choice([(1, 8), (1, 60), (1, 128), (8, 8), (4, 16), (8, 20), (3, 7), (16, 4)])
        kept = rng.randint(1, groups)
        E = groups * per
        score = rng.choice(["topk", "sigmoid", "softmax"])
        if score == "topk":
            groups, kept = 1, 1
        k = rng.randint(1, min(8, kept * per if groups > 1 else E))
        H, F = _size(rng, 128, 6144, 64), _size(rng, 64, 2048, 64)
        return {"op": op, "T": rng.randint(1, min(16, 64 * 6144 * 2048 // (k * H * F))), "E": E, "H": H, "F": F,
                "shared": rng.choice([0, 0, 64, 512, 1408]), "k": k, "score": score,
                "bias": score == "sigmoid" and rng.random() < 0.7, "groups": groups, "topk_groups": kept,
                "renorm": score == "topk" or rng.random() < 0.6, "scale": 1.0 if score == "topk" else rng.choice([1.0, 2.5])}
    if op in ("norm", "norm_bwd"):
        case = {"op": op, "T": _log(rng, 1, 8192), "H": _size(rng, 128, 6144, 16), "x": rng.choice(["bf16", "fp32"]),
                "res": rng.choice(["bf16", "fp32"]), "gate": rng.choice(["none", "channel", "token"]),
                "next": rng.random() < 0.75, "res_scale": rng.choice([1.0, 0.875, 1.5]),
                "branch_scale": rng.choice([1.0, 0.25])}
        if op == "norm_bwd":
            case["dy"] = rng.choice(["bf16", "fp32"])
        return case
    B, D = _log(rng, 1, 64), rng.randint(0, 8)
    most = 64 * 9 * 151552 // (B * (2 * D + 1))
    return {"op": op, "B": B, "D": D, "V": min(most, _log(rng, 100, 152000)), "logits": rng.choice(["bf16", "fp32"]),
            "draft": rng.choice(["none", "logits", "logits"]) if D else "none", "ragged": D > 0 and rng.random() < 0.5,
            "temperature": rng.choice(["one", "each"])}


# ------------------------------------------------------------------------------------------------------- inputs

def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _bank(g, *shape):
    """Expert weights of standard deviation 0.02, drawn bank by bank."""
    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for bank in w.view(-1, *shape[-2:]):
        bank.normal_(0.0, 0.02, generator=g)
    return w


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(c), "workspace": torch.zeros(1 << 25, dtype=torch.uint8, device="cuda")}
    return _PREPARE[c["op"]](g, s, c)


def _prepare_moe(g, s, c):
    T, E, H, F, Fs = c["T"], c["E"], c["H"], c["F"], c["shared"]
    s["x"] = _randn(g, T, H, dtype=torch.bfloat16)
    s["w_router"] = _randn(g, E, H, std=0.02, dtype=torch.bfloat16)
    s["w13"], s["w2"] = _bank(g, E, 2 * F, H), _bank(g, E, H, F)
    s["ws13"], s["ws2"] = (_bank(g, 2 * Fs, H), _bank(g, H, Fs)) if Fs else (None, None)
    s["bias"] = _randn(g, E, std=0.1) if c["bias"] else None
    return s


def _prepare_norm(g, s, c):
    T, H = c["T"], c["H"]
    s["x"] = _randn(g, T, H, std=0.5, dtype=DTYPES[c["x"]])
    s["residual"] = _randn(g, T, H, std=2.0, dtype=DTYPES[c["res"]])
    s["w_post"] = (1.0 + _randn(g, H, std=0.2)).to(torch.bfloat16)
    s["w_next"] = (1.0 + _randn(g, H, std=0.2)).to(torch.bfloat16) if c["next"] else None
    s["gate"] = None
    if c["gate"] == "channel":
        s["gate"] = (0.5 + _randn(g, H, std=0.3)).to(torch.bfloat16)
    elif c["gate"] == "token":
        s["gate"] = torch.sigmoid(_randn(g, T))
    return s


def _prepare_norm_bwd(g, s, c):
    """What a forward pass has stored, and the gradients that reach its two outputs."""
    _prepare_norm(g, s, c)
    T, H = c["T"], c["H"]
    s["stream"] = _randn(g, T, H, std=2.0, dtype=DTYPES[c["res"]])
    s["rstd_post"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
    s["rstd"] = torch.rsqrt(s["stream"].float().square().mean(-1) + EPS)
    s["dres"] = _randn(g, T, H, dtype=DTYPES[c["res"]])
    s["dy"] = _randn(g, T, H, dtype=DTYPES[c["dy"]]) if c["next"] else None
    return s


def _prepare_verify(g, s, c):
    """Logits as a head gives them, a drafter whose distribution is near the target's, and tokens drawn from it."""
    B, D, V = c["B"], c["D"], c["V"]
    z = torch.randn(B, D + 1, V, generator=g, device="cuda").mul_(2.5)
    s["logits"] = z.to(DTYPES[c["logits"]])
    s["temperature"] = None
    tau = torch.ones(B, 1, 1, device="cuda")
    if c["temperature"] == "each":
        s["temperature"] = 0.6 + 0.6 * torch.rand(B, generator=g, device="cuda")
        s["temperature"][torch.rand(B, generator=g, device="cuda") < 0.2] = 0.0
        tau = torch.where(s["temperature"] == 0, 0.1, s["temperature"]).view(B, 1, 1)
    s["noise"] = torch.empty(B, V, device="cuda").exponential_(generator=g)
    s["draft_logits"], s["draft_tokens"], s["accept_u"], s["n_draft"] = None, None, None, None
    if D:
        near = z[:, :D] + torch.randn(B, D, V, generator=g, device="cuda").mul_(0.5)
        race = torch.empty(B, D, V, device="cuda").exponential_(generator=g).log_().neg_()
        s["draft_tokens"] = (near / tau + race).argmax(-1).to(torch.int32)
        if c["draft"] == "logits":
            s["draft_logits"] = near.to(DTYPES[c["logits"]])
        s["accept_u"] = torch.rand(B, D, generator=g, device="cuda")
        if c["ragged"]:
            s["n_draft"] = torch.randint(0, D + 1, (B,), generator=g, device="cuda").to(torch.int32)
    return s


_PREPARE = {"moe": _prepare_moe, "norm": _prepare_norm, "norm_bwd": _prepare_norm_bwd, "verify": _prepare_verify}


# ------------------------------------------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](state, c)


def _own_moe(s, c):
    from serve_invariant_moe_gb300 import binding
    r = binding.moe_layer_decode(s["x"], s["w_router"], s["w13"], s["w2"], c["k"], s["workspace"], ws13=s["ws13"],
                                 ws2=s["ws2"], score=None if c["score"] == "topk" else c["score"], bias=s["bias"],
                                 n_group=c["groups"], topk_group=c["topk_groups"], renormalize=c["renorm"],
                                 scale=c["scale"], out=False, out_bf16=True)
    return {"out": r["out_bf16"], "topk_idx": r["topk_idx"]}


def _own_norm(s, c):
    from serve_invariant_moe_gb300 import binding
    r = binding.sandwich_norm(s["x"], s["w_post"], s["residual"], w_next=s["w_next"], gate=s["gate"],
                              residual_scale=c["res_scale"], branch_scale=c["branch_scale"], eps=EPS)
    return {name: r[name] for name in ("residual", "rstd_post", "rstd", "out") if r[name] is not None}


def _own_norm_bwd(s, c):
    from serve_invariant_moe_gb300 import binding
    r = binding.sandwich_norm_backward(s["dy"], s["dres"], s["x"], s["w_post"], s["rstd_post"], s["stream"],
                                       w_next=s["w_next"], rstd=s["rstd"] if c["next"] else None, gate=s["gate"],
                                       residual_scale=c["res_scale"], branch_scale=c["branch_scale"])
    return {name: r[name] for name in ("dx", "dresidual", "dw_post", "dw_next", "dgate") if r[name] is not None}


def _own_verify(s, c):
    from serve_invariant_moe_gb300 import binding
    temperature = 1.0 if s["temperature"] is None else s["temperature"]
    return binding.verify_drafts(s["logits"], s["noise"], s["workspace"], draft_tokens=s["draft_tokens"],
                                 draft_logits=s["draft_logits"], accept_u=s["accept_u"], n_draft=s["n_draft"],
                                 temperature=temperature)


_OWN = {"moe": _own_moe, "norm": _own_norm, "norm_bwd": _own_norm_bwd, "verify": _own_verify}


def _plain_choice(s, c):
    """Experts and weights of each token; the logits in 64 bits, where the choice hangs on them."""
    l = s["x"].double() @ s["w_router"].double().t()
    if c["score"] == "topk":
        top, idx = (t[:, :c["k"]] for t in torch.sort(l, dim=-1, descending=True, stable=True))
        w = torch.exp(top - top[:, :1])
        return idx, (w / w.sum(-1, keepdim=True)).float()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    key = l if s["bias"] is None else score + s["bias"]
    if c["groups"] > 1:
        byg = key.view(l.shape[0], c["groups"], -1)
        value = byg.amax(-1) if s["bias"] is None or byg.shape[-1] == 1 else byg.topk(2, dim=-1).values.sum(-1)
        kept = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        out = torch.ones_like(value, dtype=torch.bool).scatter_(1, kept, False)
        key = byg.masked_fill(out.unsqueeze(-1), -math.inf).view_as(l)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return idx, (w * c["scale"]).float()


def _swiglu(gu):
    """silu(gate) * up, held in bf16 between the two products."""
    gate, up = gu.chunk(2, dim=-1)
    return (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16).float()


def _plain_moe(s, c):
    T, k = c["T"], c["k"]
    idx, w = _plain_choice(s, c)
    x = s["x"].float()
    rows = x.repeat_interleave(k, dim=0).unsqueeze(-1)
    h = _swiglu(torch.bmm(s["w13"][idx.reshape(-1)].float(), rows).squeeze(-1))
    y = torch.bmm(s["w2"][idx.reshape(-1)].float(), h.unsqueeze(-1)).view(T, k, -1)
    out = (w.unsqueeze(-1) * y).sum(1)
    if s["ws13"] is not None:
        out = out + _swiglu(x @ s["ws13"].float().t()) @ s["ws2"].float().t()
    return {"out": out.to(torch.bfloat16), "topk_idx": idx.to(torch.int32)}


def _factor(s, c):
    """What multiplies the normalised block output, apart from its weight."""
    if s["gate"] is None:
        return c["branch_scale"]
    gate = s["gate"].float() * c["branch_scale"]
    return gate.unsqueeze(-1) if c["gate"] == "token" else gate


def _plain_norm(s, c):
    x, got = s["x"].float(), {}
    got["rstd_post"] = torch.rsqrt(x.square().mean(-1) + EPS)
    branch = x * got["rstd_post"].unsqueeze(-1) * s["w_post"].float() * _factor(s, c)
    got["residual"] = (c["res_scale"] * s["residual"].float() + branch).to(s["residual"].dtype)
    if c["next"]:
        r = got["residual"].float()
        got["rstd"] = torch.rsqrt(r.square().mean(-1) + EPS)
        got["out"] = (r * got["rstd"].unsqueeze(-1) * s["w_next"].float()).to(torch.bfloat16)
    return got


def _plain_norm_bwd(s, c):
    got = {}
    d = s["dres"].float()
    if c["next"]:
        rstd, dy = s["rstd"].unsqueeze(-1), s["dy"].float()
        n = s["stream"].float() * rstd
        t = dy * s["w_next"].float()
        d = d + rstd * (t - n * (t * n).mean(-1, keepdim=True))
        got["dw_next"] = (dy * n).sum(0)
    got["dresidual"] = (c["res_scale"] * d).to(s["residual"].dtype)
    rstd, w = s["rstd_post"].unsqueeze(-1), s["w_post"].float()
    n = s["x"].float() * rstd
    if c["gate"] == "channel":
        got["dgate"] = (c["branch_scale"] * d * n * w).sum(0)
    elif c["gate"] == "token":
        got["dgate"] = (c["branch_scale"] * d * n * w).sum(-1)
    d = d * _factor(s, c)
    got["dw_post"] = (d * n).sum(0)
    t = d * w
    got["dx"] = (rstd * (t - n * (t * n).mean(-1, keepdim=True))).to(s["x"].dtype)
    return got


def _lowest(is_it):
    """The lowest index along the last axis where is_it holds; the axis' length where it holds nowhere."""
    V = is_it.shape[-1]
    return torch.where(is_it, torch.arange(V, device=is_it.device), V).amin(-1)


def _softmax64(z, scale):
    e = torch.exp((z - z.amax(-1, keepdim=True)) * scale)
    return e / e.sum(-1, keepdim=True)


def _plain_verify(s, c):
    """In 64 bits: a token is accepted or drawn by comparing numbers that lie arbitrarily near one another."""
    B, D, V = c["B"], c["D"], c["V"]
    b = torch.arange(B, device="cuda")
    z = s["logits"].double()
    tau = torch.ones(B, device="cuda") if s["temperature"] is None else s["temperature"]
    greedy = tau == 0
    scale = (1.0 / torch.where(greedy, 1.0, tau).double()).view(B, 1, 1)
    p = _softmax64(z, scale)
    top = _lowest(z == z.amax(-1, keepdim=True))
    n = torch.zeros(B, dtype=torch.long, device="cuda")
    if D:
        x = s["draft_tokens"].long()
        px = p[:, :D].gather(-1, x.unsqueeze(-1)).squeeze(-1)
        qx = torch.ones_like(px)
        if s["draft_logits"] is not None:
            q = _softmax64(s["draft_logits"].double(), scale)
            qx = q.gather(-1, x.unsqueeze(-1)).squeeze(-1)
        ok = torch.where(greedy.unsqueeze(-1), x == top[:, :D], s["accept_u"].double() * qx < px)
        count = torch.full_like(n, D) if s["n_draft"] is None else s["n_draft"].long()
        ok &= torch.arange(D, device="cuda") < count.unsqueeze(-1)
        n = ok.long().cumprod(-1).sum(-1)
    weight = p[b, n]
    if D:
        at = n.clamp_max(D - 1)
        minus = q[b, at] if s["draft_logits"] is not None else torch.zeros_like(weight).scatter_(-1, x[b, at].unsqueeze(-1), 1.0)
        left = (weight - minus).clamp_min(0.0)
        rejected = (n < count) & (left.amax(-1) > 0)
        weight = torch.where(rejected.unsqueeze(-1), left, weight)
    race = weight / s["noise"].double()
    last = torch.where(greedy, top[b, n], _lowest(race == race.amax(-1, keepdim=True)))
    tokens = torch.full((B, D + 1), -1, dtype=torch.long, device="cuda")
    if D:
        tokens[:, :D] = torch.where(torch.arange(D, device="cuda") < n.unsqueeze(-1), x, -1)
    tokens[b, n] = last
    logp = torch.log(p.gather(-1, tokens.clamp_min(0).unsqueeze(-1)).squeeze(-1))
    logp = torch.where(tokens >= 0, logp, 0.0)
    return {"tokens": tokens.to(torch.int32), "n_accepted": n.to(torch.int32), "logp": logp.float()}


_PLAIN = {"moe": _plain_moe, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "verify": _plain_verify}


# ------------------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    op = c["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "moe":
        T, E, H, F, Fs, k = c["T"], c["E"], c["H"], c["F"], c["shared"], c["k"]
        active = E * (1.0 - (1.0 - k / E) ** T)                  # experts that some token chose, on average
        weights = 6 * H * (active * F + Fs) + 2 * E * H
        return {"bytes": int(weights + 4 * T * H + 4 * T * k), "flops": 2 * T * H * (3 * (k * F + Fs) + E)}
    if op == "norm":
        per = size[c["x"]] + 2 * size[c["res"]] + 2 * c["next"]
        return {"bytes": c["T"] * (c["H"] * per + 8) + 6 * c["H"], "flops": 12 * c["T"] * c["H"]}
    if op == "norm_bwd":
        per = 2 * size[c["x"]] + 2 * size[c["res"]] + c["next"] * (size[c["dy"]] + size[c["res"]])
        return {"bytes": c["T"] * (c["H"] * per + 8) + 16 * c["H"], "flops": 24 * c["T"] * c["H"]}
    drafts = c["D"] / 2 if c["ragged"] else c["D"]
    rows = drafts + 1 + (drafts if c["draft"] == "logits" else 0)
    return {"bytes": int(c["B"] * c["V"] * (rows * size[c["logits"]] + 4)), "flops": int(c["B"] * c["V"] * 4 * (rows + 1))}


# ------------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    with torch.no_grad():
        return _EXACT[case["op"]](prepare(case, seed), case)


def _exact_gates(s, c, logits):
    """One token's experts and their weights, from its logits."""
    l = logits.tolist()
    if c["score"] == "sigmoid":
        score = torch.sigmoid(logits).tolist()
    elif c["score"] == "softmax":
        score = torch.softmax(logits, 0).tolist()
    else:
        score = torch.exp(logits - logits.max()).tolist()
    key = l if s["bias"] is None else [a + b for a, b in zip(score, s["bias"].tolist())]
    per = c["E"] // c["groups"]
    first = 2 if s["bias"] is not None and per > 1 else 1
    value = [sum(sorted(key[g * per:(g + 1) * per], reverse=True)[:first]) for g in range(c["groups"])]
    kept = sorted(range(c["groups"]), key=lambda g: -value[g])[:c["topk_groups"]]
    experts = sorted((e for g in sorted(kept) for e in range(g * per, (g + 1) * per)), key=lambda e: -key[e])[:c["k"]]
    total = sum(score[e] for e in experts) if c["renorm"] else 1.0
    return [(e, c["scale"] * score[e] / total) for e in experts]


def _exact_expert(x, w13, w2):
    g, u = (w13.double() @ x).chunk(2)
    return w2.double() @ (g * torch.sigmoid(g) * u).to(torch.bfloat16).double()


def _exact_moe(s, c):
    x = s["x"].double()
    logits = torch.nn.functional.linear(x, s["w_router"].double())
    rows = []
    for t in range(c["T"]):
        row = sum(w * _exact_expert(x[t], s["w13"][e], s["w2"][e]) for e, w in _exact_gates(s, c, logits[t]))
        rows.append(row if s["ws13"] is None else row + _exact_expert(x[t], s["ws13"], s["ws2"]))
    return {"out": torch.stack(rows), "topk_idx": None}


def _exact_norm(s, c):
    x = s["x"].double()
    got = {"rstd_post": (torch.mean(x * x, 1) + EPS) ** -0.5}
    n = x * got["rstd_post"][:, None] * s["w_post"].double()[None]
    if s["gate"] is not None:
        n *= s["gate"].double()[:, None] if c["gate"] == "token" else s["gate"].double()[None]
    got["residual"] = s["residual"].double() * c["res_scale"] + n * c["branch_scale"]
    if c["next"]:
        r = got["residual"].float().to(s["residual"].dtype).double()        # the row as it is stored
        got["rstd"] = (torch.mean(r * r, 1) + EPS) ** -0.5
        got["out"] = r * got["rstd"][:, None] * s["w_next"].double()[None]
    return got


def _exact_rms(r, rstd, weight):
    """The norm of a row whose rstd is given, with the derivative through its mean square."""
    ms = torch.mean(r * r, 1, keepdim=True)
    rstd = rstd.double()[:, None]
    return r * (rstd - 0.5 * rstd ** 3 * (ms - ms.detach())) * weight


def _exact_norm_bwd(s, c):
    got = {}
    leaf = lambda t: t.double().requires_grad_()   # noqa: E731
    with torch.enable_grad():
        d = s["dres"].double()
        if c["next"]:
            r, w = leaf(s["stream"]), leaf(s["w_next"])
            (_exact_rms(r, s["rstd"], w) * s["dy"].double()).sum().backward()
            d = d + r.grad
            got["dw_next"] = w.grad
        x, w, res = leaf(s["x"]), leaf(s["w_post"]), leaf(s["residual"])
        n = _exact_rms(x, s["rstd_post"], w)
        if s["gate"] is not None:
            gate = leaf(s["gate"])
            n = n * (gate[:, None] if c["gate"] == "token" else gate)
        ((c["res_scale"] * res + c["branch_scale"] * n) * d).sum().backward()
    if s["gate"] is not None:
        got["dgate"] = gate.grad
    got.update(dx=x.grad, dw_post=w.grad, dresidual=res.grad)
    return got


def _exact_verify(s, c):
    """Request by request; the tokens are whole numbers, the log-probabilities of the emitted ones are not."""
    B, D = c["B"], c["D"]
    logp = torch.zeros(B, D + 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        tau = 1.0 if s["temperature"] is None else float(s["temperature"][b])
        count = D if s["n_draft"] is None else int(s["n_draft"][b])
        z = s["logits"][b].double()
        lp = torch.log_softmax(z / (tau or 1.0), -1)
        lq = None if s["draft_logits"] is None else torch.log_softmax(s["draft_logits"][b].double() / (tau or 1.0), -1)
        i, token = 0, None
        while i < count and token is None:
            x = int(s["draft_tokens"][b, i])
            if tau == 0:
                accept = bool(z[i, x] == z[i].max()) and x == int((z[i] == z[i].max()).nonzero()[0])
            else:
                accept = bool(torch.log(s["accept_u"][b, i].double()) + (0.0 if lq is None else lq[i, x]) < lp[i, x])
            if accept:
                logp[b, i] = lp[i, x]
                i += 1
                continue
            if tau != 0:
                left = torch.exp(lp[i])
                if lq is None:
                    left[x] = 0.0
                else:
                    left -= torch.exp(lq[i])
                if float(left.max()) > 0:
                    token = int((left / s["noise"][b].double()).argmax())
            break
        if tau == 0:
            token = int((z[i] == z[i].max()).nonzero()[0])
        elif token is None:
            token = int((lp[i] - torch.log(s["noise"][b].double())).argmax())
        logp[b, i] = lp[i, token]
    return {"tokens": None, "n_accepted": None, "logp": logp}


_EXACT = {"moe": _exact_moe, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "verify": _exact_verify}
