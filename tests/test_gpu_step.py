"""A drafted decode step's operators together: norms around a block, the layer of a few tokens in one kernel, the head, the
verification; the block's prefill, decode, backward and a whole step as a graph."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def layer_weights(E, H, F, Fs, k, routing=None, seed=0, std=0.05):
    from serve_invariant_moe_gb300 import api
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.empty(s, dtype=BF, device=DEV).normal_(0.0, std, generator=g)   # noqa: E731
    return api.MoEWeights(r(E, H), r(E, 2 * F, H), r(E, H, F), k, r(2 * Fs, H) if Fs else None, r(H, Fs) if Fs else None, routing)


def stack(n, H, E=32, F=128, Fs=128, k=4, fused=True, gate=True):
    """n blocks: block i's w_next is the norm before block i + 1."""
    from serve_invariant_moe_gb300.block import MoEBlock, MoEBlockWeights
    g = torch.Generator().manual_seed(5)
    w = lambda: (1 + 0.2 * torch.randn(H, generator=g)).to(BF).to(DEV)   # noqa: E731
    return [MoEBlock(MoEBlockWeights(layer_weights(E, H, F, Fs, k, seed=i), w(), w() if i + 1 < n else None,
                                     (0.5 * w()).to(BF) if gate else None, residual_scale=0.875, branch_scale=0.5), fused)
            for i in range(n)], w()


def run(blocks, w_first, x, decode):
    """x [T, H] bf16, embedded rows -> the last residual."""
    from serve_invariant_moe_gb300 import binding
    n, r = binding.add_rms_norm(x, w_first)["out"], x
    for b in blocks:
        n, r = (b.decode if decode else b.prefill)(n, r)
    return r


@pytest.mark.parametrize("T", [1, 5, 16, 17, 100])
def test_prefill_and_decode_give_the_same_bits(T):
    blocks, w = stack(3, 256)
    plain, _ = stack(3, 256, fused=False)
    x = torch.randn(T, 256, generator=torch.Generator().manual_seed(T)).to(BF).to(DEV)
    want = run(plain, w, x, decode=False)
    assert torch.equal(run(blocks, w, x, decode=True), want)
    assert torch.equal(run(blocks, w, x, decode=False), want)
    assert torch.equal(run(plain, w, x, decode=True), want)
    for b in blocks:
        b.check()


@pytest.mark.parametrize("scored", [False, True])
def test_a_fused_layer_decodes_like_the_separate_kernels(scored):
    from serve_invariant_moe_gb300 import api
    bias = 0.1 * torch.randn(32, generator=torch.Generator().manual_seed(2)).to(DEV)
    routing = api.Routing("sigmoid", bias, 4, 2, True, 2.5) if scored else None
    w = layer_weights(32, 512, 256, 128, 4, routing)
    plain, fused = api.MoELayer(w), api.MoELayer(w, fused=True)
    x = torch.randn(40, 512, device=DEV).to(BF)
    for B in (16, 3, 1, 17, 40, 5):
        bf = [torch.empty(B, 512, dtype=BF, device=DEV) for _ in range(2)]
        a, b = plain.decode(x[:B], bf[0]), fused.decode(x[:B], bf[1])
        assert torch.equal(a, b) and torch.equal(bf[0], bf[1]), B
        assert torch.equal(plain._decode["idx"][:B], fused._decode["idx"][:B])
        assert torch.equal(plain._decode["w"][:B], fused._decode["w"][:B])
        assert torch.equal(fused.prefill(x[:B]), a)
    graphs = api.DecodeGraphs(fused, buckets=(1, 4, 16, 32))
    for B in (1, 3, 16, 20):
        assert torch.equal(graphs(x[:B]), plain.decode(x[:B])), B
    fused.check()
    with pytest.raises(ValueError):
        fused.decode(x[:2].float())


def test_a_fused_layer_gets_larger_and_keeps_its_graphs():
    from serve_invariant_moe_gb300 import api
    w = layer_weights(8, 256, 128, 0, 2)
    layer, plain = api.MoELayer(w, fused=True), api.MoELayer(w)
    graphs = api.DecodeGraphs(layer, buckets=(1, 2))
    x = torch.randn(16, 256, device=DEV).to(BF)
    want = plain.decode(x).clone()
    assert torch.equal(layer.decode(x), want)                # new buffers, a larger workspace
    assert torch.equal(graphs(x[:2]), want[:2])


def test_a_drafted_step_from_embeddings_to_tokens():
    """Three requests with three drafts each through two blocks, the head and the verification, eager and as one graph; the
    drafts that the target itself would take greedily are all accepted."""
    from serve_invariant_moe_gb300 import api, binding
    B, D, H, V = 3, 3, 256, 1024
    T = B * (D + 1)
    blocks, w = stack(2, H)
    g = torch.Generator().manual_seed(11)
    w_vocab = (0.1 * torch.randn(V, H, generator=g)).to(BF).to(DEV)
    w_last = torch.ones(H, dtype=BF, device=DEV)
    x = torch.randn(T, H, generator=g).to(BF).to(DEV)
    noise = torch.empty(B, V).exponential_(generator=g).to(DEV)
    u = torch.rand(B, D, generator=g).to(DEV)
    drafts = torch.zeros(B, D, dtype=torch.int32, device=DEV)
    tau = torch.tensor([0.0, 1.0, 0.7], device=DEV)
    ws = binding.new_workspace(max(binding.workspace_size(T, H, V=V), binding.verify_workspace_size(B, D, V)))
    logits = torch.empty(B, D + 1, V, device=DEV)

    def step():
        r = run(blocks, w, x, decode=True)
        hidden = binding.add_rms_norm(r, w_last)["out"]
        return api.head_verify_drafts(hidden, w_vocab, noise, drafts, accept_u=u, temperature=tau, logits=logits, workspace=ws)
    first = step()
    drafts.copy_(first["logits"][:, :D].argmax(-1).to(torch.int32))
    got = {n: t.clone() for n, t in step().items()}
    binding.check_status(ws)
    assert got["n_accepted"][0] == D and got["tokens"][0, D] == got["logits"][0, D].argmax()
    assert torch.equal(got["logits"], first["logits"])
    # what was emitted has the head's log-probability at its temperature
    lp = torch.log_softmax(got["logits"].double() / torch.where(tau == 0, 1.0, tau).double()[:, None, None], -1)
    for b in range(B):
        for i in range(int(got["n_accepted"][b]) + 1):
            assert abs(float(got["logp"][b, i]) - float(lp[b, i, got["tokens"][b, i]])) <= 1e-4
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(5):
        logits.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(out[n], got[n]), n
    # other tokens through the same graph, against the eager step
    x.copy_(torch.randn(T, H, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: t.clone() for n, t in out.items()}
    eager = step()
    for n in replayed:
        assert torch.equal(replayed[n], eager[n]), n
    for b in blocks:
        b.check()


def test_head_verify_drafts_refuses_other_sizes():
    from serve_invariant_moe_gb300 import api
    hidden, w = torch.zeros(6, 64, dtype=BF, device=DEV), torch.zeros(256, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="rows"):
        api.head_verify_drafts(hidden, w, torch.ones(4, 256, device=DEV))
    with pytest.raises(ValueError, match="rows"):
        api.head_verify_drafts(hidden, w, torch.ones(6, 128, device=DEV))
    assert api.head_verify_drafts(hidden, w, torch.ones(6, 256, device=DEV))["tokens"].shape == (6, 1)


@pytest.mark.parametrize("gate", [False, True])
def test_the_blocks_gradients_are_its_formulas(gate):
    """One block with every expert chosen (no selection that could flip) against torch.autograd in 64 bits.  The layer's
    gradient products take bf16 operands (dy, [dg | du], h: 2^-8 of each): 2e-2 of the largest entry bounds what the existing
    backward is held to (1e-2) with the norm's gradient on top."""
    from serve_invariant_moe_gb300.block import MoEBlock, MoEBlockWeights
    T, H, E, F, k = 24, 128, 8, 128, 8
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    w = layer_weights(E, H, F, 0, k, std=0.1)
    wb = MoEBlockWeights(w, (1 + 0.2 * r(H)).to(BF).to(DEV), (1 + 0.2 * r(H)).to(BF).to(DEV),
                         (0.5 + 0.3 * r(H)).to(BF).to(DEV) if gate else None, 0.875, 0.5)
    block = MoEBlock(wb)
    n, res = r(T, H).to(BF).to(DEV), r(T, H).to(DEV)
    dn, dr = r(T, H).to(DEV), r(T, H).to(DEV)
    fwd = block.prefill(n, res, return_all=True)
    got = block.backward(fwd, dn, dr)
    leaf = lambda t: t.double().detach().requires_grad_()   # noqa: E731
    a = {name: leaf(t) for name, t in dict(n=n, res=res, w_post=wb.w_post, w_next=wb.w_next, w_router=w.w_router, w13=w.w13,
                                            w2=w.w2).items()}
    ga = leaf(wb.gate) if gate else torch.ones(H, dtype=torch.float64, device=DEV)
    gates = torch.softmax(a["n"] @ a["w_router"].T, -1)
    gu = torch.einsum("th,efh->tef", a["n"], a["w13"])
    h = torch.nn.functional.silu(gu[..., :F]) * gu[..., F:]
    m = torch.einsum("te,tef,ehf->th", gates, h, a["w2"])
    rms = lambda x: x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()   # noqa: E731
    stream = 0.875 * a["res"] + 0.5 * ga * rms(m) * a["w_post"]
    out = rms(stream) * a["w_next"]
    ((out * dn.double()).sum() + (stream * dr.double()).sum()).backward()
    want = dict(dn=a["n"].grad, dresidual=a["res"].grad, dw_post=a["w_post"].grad, dw_next=a["w_next"].grad)
    if gate:
        want["dgate"] = ga.grad
    else:
        assert got["dgate"] is None
    for name, t in want.items():
        err = (got[name].double() - t).abs().max() / t.abs().max()
        assert err <= 2e-2, (name, float(err))
    for name in ("w_router", "w13", "w2"):
        t = a[name].grad
        err = (got["layer"]["d" + name].double() - t).abs().max() / t.abs().max()
        assert err <= 2e-2, (name, float(err))


def test_a_training_step_forward_and_backward_of_two_blocks():
    """Gradients through two blocks along a random direction of the embedded rows against the difference of the loss, the
    residual stream in fp32."""
    from serve_invariant_moe_gb300 import binding
    T, H = 40, 128
    blocks, w = stack(2, H, E=8, F=128, Fs=0, k=8)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, H, generator=g).to(DEV)
    target = torch.randn(T, H, generator=g).to(DEV)

    def forward(x):
        f0 = binding.add_rms_norm(x, w)
        n, r, kept = f0["out"], x, []
        for b in blocks:
            f = b.prefill(n, r, return_all=True)
            kept.append(f)
            n, r = f["out"], f["residual"]
        return f0, kept, r
    f0, kept, r = forward(x)
    dres, dn = (r - target), None
    for b, f in zip(reversed(blocks), reversed(kept)):
        back = b.backward(f, dn, dres)
        dn, dres = back["dn"], back["dresidual"]
    dx = binding.add_rms_norm_backward(dn, x, w, f0["rstd"], dres=dres)["dx"]
    v = torch.randn(T, H, generator=g).to(DEV)
    loss = lambda x: float(0.5 * (forward(x)[2].double() - target.double()).square().sum())   # noqa: E731
    h = 0.05        # rows are rounded to bf16 on the way: a step that moves them by many roundings
    want = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
    have = float((dx.double() * v.double()).sum())
    assert np.isfinite(have) and abs(have - want) <= 0.05 * float(dx.double().norm() * v.double().norm()), (have, want)


@pytest.mark.parametrize("fused", [True, False])
def test_a_captured_block_outlives_a_larger_batch(fused):
    """A block's decode captured by its caller, then eager steps of larger batches: the graph's buffers stay its own, whatever
    is allocated afterwards, and it gives the bits of the eager step."""
    (block, _), _ = stack(2, 256, fused=fused)
    g = torch.Generator().manual_seed(21)
    x = torch.randn(40, 256, generator=g).to(BF).to(DEV)
    n, r = x[:2].clone(), x[2:4].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in block.decode(n, r)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.decode(n, r)
    sizes = [t.numel() * t.element_size() for t in block.layer._decode.values() if isinstance(t, torch.Tensor)]
    for B in (16, 40):
        block.decode(x[:B], x[:B])
    torch.cuda.synchronize()
    others = [torch.full((s,), 0x5a, dtype=torch.uint8, device=DEV) for s in sizes for _ in range(2)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(bool((t == 0x5a).all()) for t in others)
    block.check()


def test_a_step_captured_before_any_eager_one():
    """Buffers made inside the capture are the graph's: the eager steps behind it have others, whose workspaces are clear."""
    (block, _), _ = stack(2, 256)
    g = torch.Generator().manual_seed(22)
    n, r = (torch.randn(3, 256, generator=g).to(BF).to(DEV) for _ in range(2))
    other, _ = stack(2, 256)
    want = other[0].decode(n, r)                    # (also sets the kernels' attributes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.decode(n, r)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(block.decode(n, r), want))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    block.check()


def alone_and_in_two_threads(call, inputs):
    """call(*inputs[i]) has the bits of the same call alone when two threads, each on a stream of its own, repeat it."""
    want = [call(*i) for i in inputs]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = call(*inputs[i])
                stream.synchronize()
                bad.extend((i, j) for j, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("T", [8, 100])
def test_two_threads_through_one_layer(T):
    from serve_invariant_moe_gb300 import api
    layer = api.MoELayer(layer_weights(32, 256, 128, 128, 4), fused=True)
    g = torch.Generator().manual_seed(T)

    def call(x, dout):
        b = layer.backward(x, layer.prefill(x, return_all=True), dout)
        return [layer.prefill(x), *(b[name] for name in ("dx", "dw_router", "dw13", "dw2", "dws13", "dws2"))]
    alone_and_in_two_threads(call, [(torch.randn(T, 256, generator=g).to(BF).to(DEV), torch.randn(T, 256, generator=g).to(DEV))
                                    for _ in range(2)])
    layer.check()


@pytest.mark.parametrize("T", [8, 100])
def test_two_threads_through_one_block(T):
    (block, _), _ = stack(2, 256)
    g = torch.Generator().manual_seed(T)
    r = lambda: torch.randn(T, 256, generator=g).to(BF).to(DEV)   # noqa: E731

    def call(n, res, dn, dres):
        b = block.backward(block.prefill(n, res, return_all=True), dn, dres)
        return [*block.prefill(n, res), *(b[name] for name in ("dn", "dresidual", "dw_post", "dw_next", "dgate"))]
    alone_and_in_two_threads(call, [(r(), r(), r(), r()) for _ in range(2)])
    block.check()


def test_head_verify_drafts_without_a_workspace():
    """In memory of any content, with the results of a call that is given one; its status can be read."""
    from serve_invariant_moe_gb300 import api, binding
    B, D, H, V = 3, 2, 256, 1000
    g = torch.Generator().manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    args = (r(B * (D + 1), H).to(BF).to(DEV), (0.1 * r(V, H)).to(BF).to(DEV), torch.empty(B, V).exponential_(generator=g).to(DEV),
            torch.randint(0, V, (B, D), generator=g).to(torch.int32).to(DEV), None, torch.rand(B, D, generator=g).to(DEV))
    need = max(binding.workspace_size(B * (D + 1), H, V=V), binding.verify_workspace_size(B, D, V))
    ws = binding.new_workspace(need)
    want = api.head_verify_drafts(*args, workspace=ws)
    binding.check_status(ws)
    dirty = [torch.full((need,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    del dirty
    got = api.head_verify_drafts(*args)
    binding.check_status(got.pop("workspace"))
    assert set(got) == set(want) and all(torch.equal(got[n], want[n]) for n in want)


def test_a_block_of_more_experts_than_the_one_kernel_takes():
    (block, _), _ = stack(2, 128, E=600, F=128, Fs=0, fused=None)
    (plain, _), _ = stack(2, 128, E=600, F=128, Fs=0, fused=False)
    x = torch.randn(20, 128, generator=torch.Generator().manual_seed(41)).to(BF).to(DEV)
    for T in (1, 16, 20):
        want = plain.prefill(x[:T], x[:T])
        for call in (block.prefill, block.decode):
            assert all(torch.equal(a, b) for a, b in zip(call(x[:T], x[:T]), want)), T


@pytest.mark.parametrize("Fs", [0, 128])
def test_the_bf16_copy_may_go_where_the_tokens_are(Fs):
    """Over the tokens themselves or shifted over some of them: the one-kernel layer reads them to the end, so such a call takes
    the separate kernels, which give the same bits."""
    from serve_invariant_moe_gb300 import api
    w = layer_weights(32, 256, 128, Fs, 4)
    plain, fused = api.MoELayer(w), api.MoELayer(w, fused=True)
    x = torch.randn(16, 256, generator=torch.Generator().manual_seed(42)).to(BF).to(DEV)
    want = torch.empty(9, 256, dtype=BF, device=DEV)
    out = plain.prefill(x[:9], want)
    for name in ("decode", "prefill"):
        for first in (0, 3):
            y = x.clone()
            got = getattr(fused, name)(y[:9], y[first:first + 9])
            assert torch.equal(got, out) and torch.equal(y[first:first + 9], want), (name, first)
    fused.check()


def test_gradients_through_two_blocks():
    """The embedded rows' gradient through a norm and two blocks, every expert chosen, the residual stream in fp32.

    Against 64-bit autograd in the norm of the difference: each block's backward is held to 2e-2 (its products take bf16
    operands), two of them to 4e-2.  Against the difference of the loss along the gradient itself, whole and restricted to some
    rows or columns: there the product with the gradient is |dx|^2, so that 5 % of it is an error of 5 %.  A step moves every
    element by 0.05, tens of the roundings on the way (2^-9 of a value), whose sum over thousands of elements is far below
    1 %; the third derivative's share is (0.05)^2 / 6 of it."""
    from serve_invariant_moe_gb300 import binding
    T, H, F = 40, 128, 128
    blocks, w = stack(2, H, E=8, F=F, Fs=0, k=8)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, H, generator=g).to(DEV)
    target = torch.randn(T, H, generator=g).to(DEV)

    def forward(x):
        f0 = binding.add_rms_norm(x, w)
        n, r, kept = f0["out"], x, []
        for b in blocks:
            f = b.prefill(n, r, return_all=True)
            kept.append(f)
            n, r = f["out"], f["residual"]
        return f0, kept, r
    f0, kept, r = forward(x)
    dres, dn = (r - target), None
    for b, f in zip(reversed(blocks), reversed(kept)):
        back = b.backward(f, dn, dres)
        dn, dres = back["dn"], back["dresidual"]
    dx = binding.add_rms_norm_backward(dn, x, w, f0["rstd"], dres=dres)["dx"].double()

    rms = lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt()   # noqa: E731
    leaf = x.double().requires_grad_()
    n, r = rms(leaf) * w.double(), leaf
    for b in blocks:
        l = b.w.layer
        gu = torch.einsum("th,efh->tef", n, l.w13.double())
        h = torch.nn.functional.silu(gu[..., :F]) * gu[..., F:]
        m = torch.einsum("te,tef,ehf->th", torch.softmax(n @ l.w_router.double().T, -1), h, l.w2.double())
        r = b.w.residual_scale * r + b.w.branch_scale * b.w.gate.double() * rms(m) * b.w.w_post.double()
        n = None if b.w.w_next is None else rms(r) * b.w.w_next.double()
    (0.5 * (r - target.double()).square().sum()).backward()
    assert (dx - leaf.grad).norm() <= 4e-2 * leaf.grad.norm()

    loss = lambda x: float(0.5 * (forward(x)[2].double() - target.double()).square().sum())   # noqa: E731
    mask = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for rows_, cols in ((slice(None), slice(None)), (slice(0, 7), slice(None)), (slice(20, 40), slice(0, 64)),
                        (slice(None), slice(100, 128))):
        mask.zero_()
        mask[rows_, cols] = 1
        v = dx * mask
        v = v / (v.norm() / mask.sum().sqrt())
        step = (0.05 * v).float()
        want = (loss(x + step) - loss(x - step)) / 0.1
        have = float((dx * v).sum())
        assert have > 0 and abs(have - want) <= 0.05 * have, (have, want)
