"""The 8-bit block and the layer with a scored router, forward and backward, end to end.

Block: every stage is compared with a 64-bit computation on the kernel's own input of that stage (the stages' own tests
hold the tolerances), then out with the whole 64-bit composition from the dequantised operands.  Normwise per token: the
e4m3 rounding of the norm's output and of h (2^-4 relative at most, both present on the two sides only up to boundary
flips) is shared, so what differs is flips, each moving one of K terms by 2^-3 of itself: 1e-2 covers them.
"""
import numpy as np
import pytest
import torch

from helpers import MOE_MAX_REL, MOE_MEAN_REL, dot_bound, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def make_block(E=16, H=320, F=256, k=4, Fs=128, seed=0, **routing):
    from serve_invariant_moe_gb300 import api, block
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).to(DEV)   # noqa: E731
    routing = dict(score="sigmoid", bias=(torch.randn(E, generator=g) * 0.1).to(DEV), n_group=4, topk_group=2,
                   scale=2.5) | routing
    w = block.Fp8MoEWeights.from_bf16((1 + n(H, std=0.2)).to(torch.bfloat16), n(E, H, std=0.1), n(E, 2 * F, H), n(E, H, F), k,
                                      api.Routing(**routing), n(2 * Fs, H) if Fs else None, n(H, Fs) if Fs else None)
    return block.Fp8MoEBlock(w)


def tokens(T, H, seed=1, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed + T)
    return torch.randn(T, H, generator=g).to(dtype).to(DEV), torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)


def deq(q, s):
    return q.double() * s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]


def deq_w(q, s):
    full = s.double().repeat_interleave(128, -2)[..., :q.shape[-2], :].repeat_interleave(128, -1)[..., :q.shape[-1]]
    return q.double() * full


def quantised(y):
    T, K = y.shape
    b = torch.nn.functional.pad(y, (0, -K % 128)).view(T, -1, 128)
    s = (b.abs().amax(-1, keepdim=True) / 448).clamp_min(2.0 ** -126)
    return ((b / s).float().to(torch.float8_e4m3fn).double() * s).view(T, -1)[:, :K]


def expert(n, w13, w2):
    g, u = (n @ w13.T).chunk(2, dim=-1)
    return quantised(g * torch.sigmoid(g) * u) @ w2.T


@pytest.mark.parametrize("T", [1, 7, 64, 300])
@pytest.mark.parametrize("Fs", [0, 128])
def test_block_matches_64_bits(T, Fs):
    blk = make_block(Fs=Fs)
    w = blk.w
    x, res = tokens(T, w.H)
    r = blk.prefill(x, res, return_all=True)
    from serve_invariant_moe_gb300 import binding
    binding.check_status(r["workspace"])
    new_res = (x + res.float()).to(torch.bfloat16)
    assert torch.equal(r["residual"], new_res)
    rr = new_res.double()
    norm = rr / (rr.square().mean(-1, keepdim=True) + w.eps).sqrt() * w.w_norm.double()
    assert rel_err(r["norm"].double().cpu().numpy(), norm.cpu().numpy()).max() < 5e-3
    n8 = deq(r["q"], r["q_scale"])                       # the experts' input as the kernels have it
    assert rel_err(n8.cpu().numpy(), norm.cpu().numpy()).max() < 2.0 ** -4
    out = torch.zeros(T, w.H, dtype=torch.float64, device=DEV)
    idx, gate = r["topk_idx"].long(), r["topk_w"].double()
    for e in range(w.E):
        y = expert(n8, deq_w(w.w13[e], w.w13_scale[e]), deq_w(w.w2[e], w.w2_scale[e]))
        out += (gate * (idx == e)).sum(-1, keepdim=True) * y
    if Fs:
        out += expert(n8, deq_w(w.ws13[0], w.ws13_scale[0]), deq_w(w.ws2[0], w.ws2_scale[0]))
    err = rel_err(r["out"].double().cpu().numpy(), out.cpu().numpy())
    assert err.max() <= MOE_MAX_REL and err.mean() <= MOE_MEAN_REL


def test_prefill_decode_and_graph_give_the_same_bits():
    from serve_invariant_moe_gb300 import block
    blk = make_block(E=32, H=512, F=384, k=6, n_group=8, topk_group=3)
    x, res = tokens(400, 512, dtype=torch.bfloat16)
    out, new = blk.prefill(x, res)
    for rows in ([5], [5, 17, 399], list(range(100, 180))):
        o, n = blk.decode(x[rows].contiguous(), res[rows].contiguous())
        assert torch.equal(o, out[rows]) and torch.equal(n, new[rows])
    blk.check()
    g = block.Fp8DecodeGraph(blk, 3)
    for rows in ([1, 2, 3], [300, 0, 64]):
        g.x.copy_(x[rows])
        g.residual.copy_(res[rows])
        o, n = g.replay()
        assert torch.equal(o, out[rows]) and torch.equal(n, new[rows])


def test_block_without_a_residual_and_on_another_stream():
    blk = make_block(Fs=0)
    x, _ = tokens(33, blk.w.H, dtype=torch.bfloat16)
    want, res = blk.prefill(x)
    assert res is x
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = blk.prefill(x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_block_without_tokens():
    blk = make_block()
    out, res = blk.prefill(torch.empty(0, blk.w.H, device=DEV), torch.empty(0, blk.w.H, dtype=torch.bfloat16, device=DEV))
    assert out.shape == (0, blk.w.H) and res.shape == (0, blk.w.H)


ROUTINGS = [dict(score="sigmoid", scale=2.5), dict(score="sigmoid", n_group=4, topk_group=2, renormalize=False),
            dict(score="softmax", renormalize=False), dict(score="softmax", renormalize=True)]


def routed_layer(routing, E=16, H=192, F=128, k=3, Fs=128, seed=3):
    from serve_invariant_moe_gb300 import api
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=0.05: (torch.randn(*s, generator=g) * std).to(torch.bfloat16).to(DEV)   # noqa: E731
    routing = dict(routing)
    if routing["score"] == "sigmoid":
        routing["bias"] = (torch.randn(E, generator=g) * 0.1).to(DEV)
    w = api.MoEWeights(n(E, H, std=0.1), n(E, 2 * F, H), n(E, H, F), k, n(2 * Fs, H) if Fs else None,
                       n(H, Fs) if Fs else None, api.Routing(**routing))
    return api.MoELayer(w)


def routed_ref(layer, x, idx):
    """The layer in 64 bits with the choice given; h rounded to bf16."""
    w = layer.w
    r = w.routing
    x = x.double()

    def ffn(w13, w2):
        g, u = (x @ w13.double().T).chunk(2, dim=-1)
        return (g * torch.sigmoid(g) * u).to(torch.bfloat16).double() @ w2.double().T
    l = x @ w.w_router.double().T
    s = torch.sigmoid(l) if r.score == "sigmoid" else torch.softmax(l, -1)
    gate = s.gather(1, idx.long())
    if r.renormalize:
        gate = gate / gate.sum(-1, keepdim=True)
    gate = gate * r.scale
    out = ffn(w.ws13, w.ws2) if w.ws13 is not None else 0.0
    for e in range(w.E):
        out = out + (gate * (idx == e)).sum(-1, keepdim=True) * ffn(w.w13[e], w.w2[e])
    return out


@pytest.mark.parametrize("routing", ROUTINGS)
@pytest.mark.parametrize("T", [1, 50, 260])
def test_routed_layer_forward(routing, T):
    layer = routed_layer(routing)
    x, _ = tokens(T, layer.w.H, dtype=torch.bfloat16)
    fwd = layer.prefill(x, return_all=True)
    out = routed_ref(layer, x, fwd["topk_idx"])
    err = rel_err(fwd["out"].double().cpu().numpy(), out.cpu().numpy())
    assert err.max() <= MOE_MAX_REL and err.mean() <= MOE_MEAN_REL


@pytest.mark.parametrize("routing", ROUTINGS)
@pytest.mark.parametrize("T", [1, 50, 260])
def test_routed_layer_backward(routing, T):
    """The experts' gradients are the very calls of the softmax top-k layer on this layer's weights and plan; the router's
    part, which is new, is compared with 64 bits on the kernel's own dgate and dxp."""
    from serve_invariant_moe_gb300 import api, binding
    layer = routed_layer(routing, Fs=0)
    w = layer.w
    x, _ = tokens(T, w.H, dtype=torch.bfloat16)
    fwd = layer.prefill(x, return_all=True)
    dout = torch.randn(T, w.H, generator=torch.Generator().manual_seed(T)).to(DEV)
    got = layer.backward(x, fwd, dout)
    top_k = api.MoELayer(api.MoEWeights(w.w_router, w.w13, w.w2, w.k)).backward(x, fwd, dout)
    for name in ("dgate", "dy", "dxp", "dw13", "dw2"):
        assert torch.equal(got[name], top_k[name]), name
    # dlogits: the formula's gradient of sum(dgate * weights), rounded to bf16 (2^-8 relative covers rounding and flips)
    r = w.routing
    l = fwd["logits"].double().requires_grad_()
    s = torch.sigmoid(l) if r.score == "sigmoid" else torch.softmax(l, -1)
    gate = s.gather(1, fwd["topk_idx"].long())
    gate = r.scale * (gate / gate.sum(-1, keepdim=True) if r.renormalize else gate)
    (gate * got["dgate"].double()).sum().backward()
    d = torch.empty(T, w.E, dtype=torch.bfloat16, device=DEV)
    binding.moe_route_select_backward(fwd["logits"], fwd["topk_idx"], got["dgate"], r.score, r.renormalize, r.scale,
                                      dlogits=False, dlogits_bf16=d)
    size = l.grad.abs().amax(-1, keepdim=True)
    assert ((d.double() - l.grad).abs() <= 2.0 ** -8 * l.grad.abs() + 1e-5 * size).all()
    # the two products from that bf16 gradient, and the sum over the token's slots
    D, X, W = d.double().cpu().numpy(), x.double().cpu().numpy(), w.w_router.double().cpu().numpy()
    assert (np.abs(got["dw_router"].double().cpu().numpy() - D.T @ X) <= dot_bound(D.T, X.T, T)).all()
    slot_row = fwd["plan"][2 * w.E + 1 + T * w.k:].view(T, w.k).long()
    slots = got["dxp"].double()[slot_row].cpu().numpy()
    tol = dot_bound(D, W.T, w.E) + (w.k + 1) * 2.0 ** -23 * (np.abs(slots).sum(1) + np.abs(D) @ np.abs(W))
    assert (np.abs(got["dx"].double().cpu().numpy() - (D @ W + slots.sum(1))) <= tol).all()


def test_routed_layer_prefill_and_decode_bits():
    from serve_invariant_moe_gb300 import api
    layer = routed_layer(ROUTINGS[0], E=32, k=4)
    x, _ = tokens(1500, layer.w.H, dtype=torch.bfloat16)
    want = layer.prefill(x)
    rows = [0, 77, 1499]
    assert torch.equal(layer.decode(x[rows].contiguous()), want[rows])
    assert torch.equal(layer.prefill(x[rows].contiguous()), want[rows])
    graphs = api.DecodeGraphs(layer, buckets=(1, 4))
    assert torch.equal(graphs(x[rows].contiguous()), want[rows])
    with pytest.raises(ValueError, match="replay"):
        layer.prefill(x, replay_idx=torch.zeros(1500, 4, dtype=torch.int32, device=DEV))


def test_softmax_routing_agrees_with_the_top_k_router():
    """softmax over all experts renormalised over the chosen = softmax over the chosen: same choice, weights to 1e-6."""
    from serve_invariant_moe_gb300 import binding
    layer = routed_layer(dict(score="softmax"))
    x, _ = tokens(200, layer.w.H, dtype=torch.bfloat16)
    fwd = layer.prefill(x, return_all=True)
    w = layer.w
    ws = binding.new_workspace(binding.workspace_size(200, w.H, w.E, w.k))
    ref = binding.moe_route_topk(x, w.w_router, w.k, ws)
    assert torch.equal(fwd["logits"], ref["logits"]) and torch.equal(fwd["topk_idx"], ref["topk_idx"])
    assert torch.equal(fwd["plan"], ref["plan"]) and torch.equal(fwd["xp"], ref["xp"])
    assert np.allclose(fwd["topk_w"].cpu().numpy(), ref["topk_w"].cpu().numpy(), rtol=1e-6, atol=0)


def test_a_captured_decode_outlives_a_larger_batch():
    """A step captured by its caller, then eager steps of larger batches: the graph's buffers stay its own."""
    block = make_block()
    H = block.w.H
    x, res = tokens(40, H, dtype=torch.bfloat16)
    n, r = x[:2].clone(), res[:2].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in block.decode(n, r)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.decode(n, r)
    sizes = [t.numel() * t.element_size() for t in block._bufs.values() if isinstance(t, torch.Tensor)]
    for B in (16, 40):
        block.decode(x[:B].contiguous(), res[:B].contiguous())
    torch.cuda.synchronize()
    others = [torch.full((s,), 0x5a, dtype=torch.uint8, device=DEV) for s in sizes for _ in range(2)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(bool((t == 0x5a).all()) for t in others)
    block.check()
