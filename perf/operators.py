"""Cases for measuring the 8-bit MoE block's operators, each with a plain form.

Three operators, in the order a block runs them:

  norm    residual addition + RMSNorm, output in bf16 and in e4m3 with a scale per row and 128 columns; its backward
  route   expert scores (sigmoid or softmax), balance bias, expert groups, top-k, renormalised weights; its backward
  gemm    e4m3 matrix product with a scale per 1 x 128 of A and 128 x 128 of B: dense, grouped gate/up with a SwiGLU
          epilogue that re-quantises its output ("swiglu"), grouped down projection in fp32 ("down")

`own` chooses between the plain forms here (elementary torch operations in 32 bits) and the framework's entry points.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------------- cases

def listed():
    glm = {"E": 256, "H": 6144, "F": 2048, "k": 8}
    qwen = {"E": 128, "H": 2048, "F": 768, "k": 8}
    return [
        # one decode step of 8 requests through a 256-expert router: latency only
        {"name": "route_decode", "op": "route", "T": 8, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 1,
         "topk_groups": 1, "renorm": True, "scale": 2.5},
        # a prefill step, group-limited choice
        {"name": "route_prefill_groups", "op": "route", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "renorm": True, "scale": 2.5},
        # a prefill step of the 128-expert layer, softmax over all experts, weights not renormalised
        {"name": "route_prefill_softmax", "op": "route", "T": 4096, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "renorm": False, "scale": 1.0},
        # the trainer's side of the prefill step
        {"name": "route_backward", "op": "route_bwd", "T": 8192, "E": 256, "k": 8, "score": "sigmoid", "renorm": True,
         "scale": 2.5},
        # one token entering the block: latency only
        {"name": "norm_decode", "op": "norm", "T": 1, "H": 6144, "x": "bf16", "res": "bf16", "out": True, "fp8": True},
        # a prefill step: the MoE layer's fp32 output added to a bf16 residual stream
        {"name": "norm_prefill", "op": "norm", "T": 8192, "H": 6144, "x": "fp32", "res": "bf16", "out": True, "fp8": True},
        # the trainer's side for the 2048-wide layer
        {"name": "norm_backward", "op": "norm_bwd", "T": 4096, "H": 2048, "x": "bf16", "dy": "fp32", "dres": True},
        # one decode step of 8 requests through a dense projection: weights are read once
        {"name": "gemm_decode", "op": "gemm", "M": 8, "N": 4096, "K": 6144, "out": "bf16"},
        # a prefill step through the same projection
        {"name": "gemm_prefill", "op": "gemm", "M": 8192, "N": 4096, "K": 6144, "out": "bf16"},
        # one decode step of 4 requests: gate/up of about 32 of 256 experts
        {"name": "swiglu_decode", "op": "swiglu", "T": 4, **glm, "skew": 0.0, "empty": 0},
        # a prefill step of the GLM-scale layer
        {"name": "swiglu_prefill", "op": "swiglu", "T": 8192, **glm, "skew": 0.0, "empty": 0},
        # a prefill step of the Qwen-like layer, skewed popularity and 8 experts without a token
        {"name": "down_skewed", "op": "down", "T": 4096, **qwen, "skew": 0.3, "empty": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, step):
    n = max(lo, _log(rng, lo, hi) // step * step)
    return n + step if n == 3072 else n      # only sizes that the configurations here have, or generic ones


def draw(rng):
    op = rng.choice(["route", "route_bwd", "norm", "norm_bwd", "gemm", "gemm", "swiglu", "down"])
    if op in ("route", "route_bwd"):
        groups, per = rng.choice([(1, 8), (1, 60), (1, 128), (1, 256), (1, 160), (1, 384), (8, 32), (4, 16), (8, 20), (3, 7),
                                  (16, 32)])
        E = groups * per
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(12, kept * per))
        score = rng.choice(["sigmoid", "softmax"])
        case = {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": k, "score": score, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            case.update(bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, topk_groups=kept)
        return case
    if op in ("norm", "norm_bwd"):
        case = {"op": op, "T": _log(rng, 1, 8192), "H": _size(rng, 128, 8192, 16), "x": rng.choice(["bf16", "fp32"])}
        if op == "norm":
            out = rng.random() < 0.6
            case.update(res=rng.choice(["bf16", "fp32", "none"]), out=out, fp8=not out or rng.random() < 0.6)
        else:
            case.update(dy=rng.choice(["bf16", "fp32"]), dres=rng.random() < 0.5)
        return case
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _size(rng, 100, 6144, 1), "K": _size(rng, 128, 8192, 16),
                "out": rng.choice(["bf16", "fp32"])}
    E = rng.choice([8, 32, 60, 128])
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, 8), "H": _size(rng, 256, 4096, 16),
            "F": _size(rng, 128, 2048, 128), "skew": rng.choice([0.0, 0.3]), "empty": rng.choice([0, 0, E // 8])}


# ------------------------------------------------------------------------------------------------------- inputs

def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _activations(g, M, K):
    """Rows as a norm would quantise them: normal values, a block's largest one at 448, scales that vary by row."""
    nb = (K + 127) // 128
    q = _randn(g, M, K, std=140.0).clamp_(-FP8_MAX, FP8_MAX).to(FP8)
    scale = torch.rand(M, nb, generator=g, device="cuda").add_(0.5).mul_(1.0 / 140.0)
    return q, scale


def _weights(g, *shape):
    """Weights of standard deviation about 0.02, a scale per block of 128 x 128; drawn bank by bank."""
    q = torch.empty(shape, dtype=FP8, device="cuda")
    for bank in q.view(-1, *shape[-2:]):
        t = torch.randn(bank.shape, generator=g, device="cuda", dtype=torch.bfloat16)
        bank.copy_(t.mul_(120.0).clamp_(-FP8_MAX, FP8_MAX))
    blocks = (*shape[:-2], (shape[-2] + 127) // 128, (shape[-1] + 127) // 128)
    scale = torch.rand(blocks, generator=g, device="cuda").add_(0.5).mul_(0.02 / 120.0)
    return q, scale


def _dispatch(g, c):
    """The plan counts | offsets | row_token | slot_row of a routed batch, with its host-side sizes."""
    T, E, k = c["T"], c["E"], c["k"]
    live = E - c["empty"]
    k = min(k, live)
    pop = -c["skew"] * 1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    pop = pop[torch.randperm(E, generator=g, device="cuda")]
    if c["empty"]:
        pop[torch.randperm(E, generator=g, device="cuda")[:c["empty"]]] = -1e9
    idx = (_randn(g, T, E, std=1.5) + pop).topk(k, dim=-1).indices
    flat = idx.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    slot_row = torch.empty_like(order)
    slot_row[order] = torch.arange(T * k, device="cuda")
    plan = torch.cat([counts, offsets, order // k, slot_row]).to(torch.int32)
    return {"plan": plan, "k": k, "rows": T * k, "active": counts.nonzero().reshape(-1), "most": int(counts.max())}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": dict(c)}
    op = c["op"]
    if op in ("route", "route_bwd"):
        s["logits"] = _randn(g, c["T"], c["E"], std=1.5)
    if op == "route":
        s["bias"] = _randn(g, c["E"], std=0.1) if c["bias"] else None
    elif op == "route_bwd":
        s["topk_idx"] = (s["logits"] + _randn(g, c["E"], std=0.3)).topk(c["k"], dim=-1).indices.to(torch.int32)
        s["dw"] = _randn(g, c["T"], c["k"])
    elif op == "norm":
        s["x"] = _randn(g, c["T"], c["H"], dtype=DTYPES[c["x"]])
        s["res"] = None if c["res"] == "none" else _randn(g, c["T"], c["H"], std=2.0, dtype=DTYPES[c["res"]])
        s["weight"] = (1.0 + _randn(g, c["H"], std=0.2)).to(torch.bfloat16)
    elif op == "norm_bwd":
        s["x"] = _randn(g, c["T"], c["H"], std=2.0, dtype=DTYPES[c["x"]])
        s["weight"] = (1.0 + _randn(g, c["H"], std=0.2)).to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
        s["dy"] = _randn(g, c["T"], c["H"], dtype=DTYPES[c["dy"]])
        s["dres"] = _randn(g, c["T"], c["H"], dtype=DTYPES[c["x"]]) if c["dres"] else None
    elif op == "gemm":
        s["a"], s["a_scale"] = _activations(g, c["M"], c["K"])
        s["b"], s["b_scale"] = _weights(g, c["N"], c["K"])
    else:
        s.update(_dispatch(g, c))
        rows, cols = (2 * c["F"], c["H"]) if op == "swiglu" else (c["H"], c["F"])
        s["a"], s["a_scale"] = _activations(g, s["rows"], cols)
        s["b"], s["b_scale"] = _weights(g, c["E"], rows, cols)
    s["workspace"] = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    return (_OWN if own else _PLAIN)[c["op"]](state, c)


def _own_route(s, c):
    from serve_invariant_moe_gb300 import binding
    r = binding.moe_route_select(s["logits"], c["k"], score=c["score"], bias=s["bias"], n_group=c["groups"],
                                 topk_group=c["topk_groups"], renormalize=c["renorm"], scale=c["scale"])
    return {"topk_idx": r["topk_idx"], "topk_w": r["topk_w"]}


def _own_route_bwd(s, c):
    from serve_invariant_moe_gb300 import binding
    return {"dlogits": binding.moe_route_select_backward(s["logits"], s["topk_idx"], s["dw"], score=c["score"],
                                                         renormalize=c["renorm"], scale=c["scale"])}


def _own_norm(s, c):
    from serve_invariant_moe_gb300 import binding
    r = binding.add_rms_norm(s["x"], s["weight"], residual=s["res"], eps=EPS, out=c["out"], fp8=c["fp8"])
    return {name: r[name] for name in ("residual", "rstd", "out", "q", "scale") if r[name] is not None}


def _own_norm_bwd(s, c):
    from serve_invariant_moe_gb300 import binding
    return binding.add_rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dres=s["dres"])


def _own_gemm(s, c):
    from serve_invariant_moe_gb300 import binding
    return {"out": binding.fp8_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"], s["workspace"],
                                    out_dtype=DTYPES[c["out"]])}


def _own_swiglu(s, c):
    from serve_invariant_moe_gb300 import binding
    return binding.moe_grouped_swiglu_fp8(s["a"], s["a_scale"], s["plan"], s["b"], s["b_scale"], c["T"], s["k"],
                                          s["workspace"])


def _own_down(s, c):
    from serve_invariant_moe_gb300 import binding
    return {"y": binding.moe_grouped_down_fp8(s["a"], s["a_scale"], s["plan"], s["b"], s["b_scale"], c["T"], s["k"],
                                              s["workspace"])}


_OWN = {"route": _own_route, "route_bwd": _own_route_bwd, "norm": _own_norm, "norm_bwd": _own_norm_bwd,
        "gemm": _own_gemm, "swiglu": _own_swiglu, "down": _own_down}


def _scores(l, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_route(s, c):
    l = s["logits"]
    score = _scores(l, c["score"])
    choice = l if s["bias"] is None else score + s["bias"]
    if c["groups"] > 1:
        byg = choice.view(l.shape[0], c["groups"], -1)
        value = byg.amax(-1) if s["bias"] is None or byg.shape[-1] == 1 else byg.topk(2, dim=-1).values.sum(-1)
        kept = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        out = torch.ones_like(value, dtype=torch.bool).scatter_(1, kept, False)
        choice = byg.masked_fill(out.unsqueeze(-1), -math.inf).view_as(l)
    idx = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"topk_idx": idx.to(torch.int32), "topk_w": w * c["scale"]}


def _plain_route_bwd(s, c):
    l, idx, dw = s["logits"], s["topk_idx"].long(), s["dw"] * c["scale"]
    p = _scores(l, c["score"])
    w = p.gather(1, idx)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        dw = (dw - (dw * w).sum(-1, keepdim=True) / total) / total
    if c["score"] == "sigmoid":
        return {"dlogits": torch.zeros_like(l).scatter_(1, idx, dw * w * (1.0 - w))}
    if c["renorm"]:
        return {"dlogits": torch.zeros_like(l).scatter_(1, idx, dw * w)}
    return {"dlogits": p * (torch.zeros_like(l).scatter_(1, idx, dw) - (dw * w).sum(-1, keepdim=True))}


def _quantised(y):
    """e4m3 values and the scale of each row's blocks of 128 columns."""
    M, K = y.shape
    nb = (K + 127) // 128
    blocks = torch.nn.functional.pad(y, (0, nb * 128 - K)).view(M, nb, 128)
    scale = (blocks.abs().amax(-1) / FP8_MAX).clamp_min(TINY)
    q = (blocks * (1.0 / scale).unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(FP8)
    return q.view(M, nb * 128)[:, :K].contiguous(), scale


def _plain_norm(s, c):
    r, got = s["x"].float(), {}
    if s["res"] is not None:
        got["residual"] = (r + s["res"].float()).to(s["res"].dtype)
        r = got["residual"].float()
    rstd = torch.rsqrt(r.square().mean(-1) + EPS)
    y = r * rstd.unsqueeze(-1) * s["weight"].float()
    got["rstd"] = rstd
    if c["out"]:
        got["out"] = y.to(torch.bfloat16)
    if c["fp8"]:
        got["q"], got["scale"] = _quantised(y)
    return got


def _plain_norm_bwd(s, c):
    r, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"].unsqueeze(-1)
    n = r * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0)}


def _spread(scale, rows, cols, block_rows):
    """A block scale at each element's place."""
    if block_rows > 1:
        scale = scale.repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return scale.repeat_interleave(128, dim=-1)[..., :cols]


def _plain_gemm(s, c):
    a = s["a"].float() * _spread(s["a_scale"], c["M"], c["K"], 1)
    b = s["b"].float() * _spread(s["b_scale"], c["N"], c["K"], 128)
    return {"out": (a @ b.t()).to(DTYPES[c["out"]])}


def _plain_grouped(s, c, rows, cols):
    """Each expert's rows times its weights: the experts with rows as one batched product over padded rows."""
    E, active, most = c["E"], s["active"], s["most"]
    counts, offsets = s["plan"][:E].long(), s["plan"][E:2 * E].long()
    a = s["a"].float() * _spread(s["a_scale"], s["rows"], cols, 1)
    at = offsets[active].unsqueeze(1) + torch.arange(most, device="cuda")
    b = s["b"][active].float() * _spread(s["b_scale"][active], rows, cols, 128)
    out = torch.bmm(a[at.clamp_max(s["rows"] - 1)], b.transpose(1, 2))
    expert = torch.repeat_interleave(torch.arange(active.numel(), device="cuda"), counts[active], output_size=s["rows"])
    within = torch.arange(s["rows"], device="cuda") - offsets[active][expert]
    return out[expert, within]


def _plain_swiglu(s, c):
    gu = _plain_grouped(s, c, 2 * c["F"], c["H"])
    gate, up = gu[:, :c["F"]], gu[:, c["F"]:]
    h, h_scale = _quantised(gate / (1.0 + torch.exp(-gate)) * up)
    return {"h": h, "h_scale": h_scale}


def _plain_down(s, c):
    return {"y": _plain_grouped(s, c, c["H"], c["F"])}


_PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
          "gemm": _plain_gemm, "swiglu": _plain_swiglu, "down": _plain_down}


# ------------------------------------------------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    op = c["op"]
    size = {"bf16": 2, "fp32": 4, "none": 0}
    if op == "route":
        return {"bytes": c["T"] * (4 * c["E"] + 8 * c["k"]) + 4 * c["E"] * c["bias"], "flops": 8 * c["T"] * c["E"]}
    if op == "route_bwd":
        dense = c["score"] == "softmax" and not c["renorm"]
        read = c["E"] if c["score"] == "softmax" else c["k"]     # sigmoid scores are needed at the chosen experts alone
        return {"bytes": 4 * c["T"] * (read + c["E"] + 2 * c["k"]), "flops": c["T"] * (8 * c["E"] if dense else 12 * c["k"])}
    if op == "norm":
        per = size[c["x"]] + 2 * size[c["res"]] + 2 * c["out"] + (1 + 4 / 128) * c["fp8"]
        return {"bytes": int(c["T"] * (c["H"] * per + 4) + 2 * c["H"]), "flops": 8 * c["T"] * c["H"]}
    if op == "norm_bwd":
        per = size[c["x"]] * (3 if c["dres"] else 2) + size[c["dy"]]
        return {"bytes": c["T"] * (c["H"] * per + 4) + 6 * c["H"], "flops": 10 * c["T"] * c["H"]}
    if op == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        nb = (K + 127) // 128
        scales = 4 * nb * (M + (N + 127) // 128)
        return {"bytes": M * K + N * K + scales + M * N * size[c["out"]], "flops": 2 * M * N * K}
    k = min(c["k"], c["E"] - c["empty"])
    S, live = c["T"] * k, c["E"] - c["empty"]
    active = live * (1.0 - (1.0 - k / live) ** c["T"])
    N, K = (2 * c["F"], c["H"]) if op == "swiglu" else (c["H"], c["F"])
    out = S * (c["F"] + 4 * (c["F"] // 128)) if op == "swiglu" else 4 * S * N
    return {"bytes": int(S * K * (1 + 4 / 128) + active * N * K + out), "flops": 2 * S * N * K}


# ------------------------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    with torch.no_grad():
        return _EXACT[case["op"]](prepare(case, seed), case)


def _exact_scores(l, kind):
    return torch.sigmoid(l) if kind == "sigmoid" else torch.softmax(l, -1)


def _exact_route(s, c):
    l = s["logits"].double()
    p = _exact_scores(l, c["score"])
    key = l.clone() if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        per = c["E"] // c["groups"]
        best = torch.sort(key.reshape(-1, c["groups"], per), dim=-1, descending=True).values
        value = best[..., 0] if s["bias"] is None or per == 1 else best[..., 0] + best[..., 1]
        order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, c["topk_groups"]:]
        key.view(-1, c["groups"], per)[torch.arange(len(l), device=l.device).unsqueeze(1), order] = -math.inf
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(p, 1, idx)
    return {"topk_idx": None, "topk_w": c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)}


def _exact_route_bwd(s, c):
    l = s["logits"].double().requires_grad_()
    with torch.enable_grad():
        w = torch.gather(_exact_scores(l, c["score"]), 1, s["topk_idx"].long())
        w = c["scale"] * (w / w.sum(1, keepdim=True) if c["renorm"] else w)
        (w * s["dw"].double()).sum().backward()
    return {"dlogits": l.grad}


def _exact_fp8(y):
    q, scale = torch.empty(y.shape, dtype=FP8, device=y.device), []
    for j in range(0, y.shape[1], 128):
        t = torch.clamp(y[:, j:j + 128].abs().max(1, keepdim=True).values / FP8_MAX, min=TINY)
        q[:, j:j + 128] = (y[:, j:j + 128] / t).float().to(FP8)
        scale.append(t)
    return q, torch.cat(scale, 1)


def _exact_norm(s, c):
    r, got = s["x"].double(), {}
    if s["res"] is not None:
        r = r + s["res"].double()
        got["residual"] = r
        r = r.float().to(s["res"].dtype).double()
    got["rstd"] = (torch.mean(r * r, 1) + EPS) ** -0.5
    y = r * got["rstd"][:, None] * s["weight"].double()
    if c["out"]:
        got["out"] = y
    if c["fp8"]:
        got["q"], got["scale"] = _exact_fp8(y)
    return got


def _exact_norm_bwd(s, c):
    r = s["x"].double().requires_grad_()
    weight = s["weight"].double().requires_grad_()
    rstd = s["rstd"].double()[:, None]
    with torch.enable_grad():
        # rstd as given, its derivative through the mean square
        inv = rstd - 0.5 * rstd ** 3 * (torch.mean(r * r, 1, keepdim=True) - torch.mean(r * r, 1, keepdim=True).detach())
        y = r * inv * weight
        (y * s["dy"].double()).sum().backward()
    dx = r.grad if s["dres"] is None else r.grad + s["dres"].double()
    return {"dx": dx, "dweight": weight.grad}


def _exact_weight(q, scale):
    i, j = (torch.arange(n, device=q.device) // 128 for n in q.shape)
    return q.double().mul_(scale.double()[i][:, j])


def _exact_rows(q, scale):
    a = q.double()
    for j in range(scale.shape[1]):
        a[:, 128 * j:128 * j + 128] *= scale[:, j:j + 1].double()
    return a


def _exact_gemm(s, c):
    return {"out": _exact_rows(s["a"], s["a_scale"]) @ _exact_weight(s["b"], s["b_scale"]).T}


def _exact_experts(s, c):
    first = s["plan"][c["E"]:2 * c["E"] + 1].tolist()
    a = _exact_rows(s["a"], s["a_scale"])
    for e in range(c["E"]):
        if first[e + 1] > first[e]:
            yield a[first[e]:first[e + 1]] @ _exact_weight(s["b"][e], s["b_scale"][e]).T


def _exact_swiglu(s, c):
    if s["rows"] * c["F"] * c["H"] > 2 ** 40:
        return None                                          # over some 20 seconds
    h = torch.cat([t[:, :c["F"]] * torch.sigmoid(t[:, :c["F"]]) * t[:, c["F"]:] for t in _exact_experts(s, c)])
    q, scale = _exact_fp8(h)
    return {"h": q, "h_scale": scale}


def _exact_down(s, c):
    return {"y": torch.cat(list(_exact_experts(s, c)))}


_EXACT = {"route": _exact_route, "route_bwd": _exact_route_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
          "gemm": _exact_gemm, "swiglu": _exact_swiglu, "down": _exact_down}
