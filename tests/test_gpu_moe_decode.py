"""The whole MoE layer of a few tokens in one kernel (moe_layer_decode): bit for bit the layer's kernels one after another, and
against 64 bits at sizes that those do not take.

Tolerance against 64 bits: a product of K bf16 terms accumulated in fp32 is within 2 K 2^-24 of the sum of its terms' absolute
values; h is rounded to bf16 (2^-8 of its value, the other side's rounding included twice that); the outputs' sums of k + 1
terms add (k + 1) 2^-24.  The choice is checked on the kernel's own logits.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def weights(E, H, F, Fs=0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + E + H + F)
    r = lambda *s: torch.empty(s, dtype=BF, device=DEV).normal_(0.0, 0.05, generator=g)   # noqa: E731
    w = dict(w_router=r(E, H), w13=r(E, 2 * F, H), w2=r(E, H, F))
    if Fs:
        w.update(ws13=r(2 * Fs, H), ws2=r(H, Fs))
    return w


def tokens(T, H, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    return torch.randn(T, H, generator=g, device=DEV).to(BF)


def space(T, w, k):
    """A workspace whose first 256 bytes are zero and whose rest is anything."""
    from serve_invariant_moe_gb300 import binding
    E, F2, H = w["w13"].shape
    Fs = w["ws13"].shape[0] // 2 if "ws13" in w else 0
    n = binding.moe_decode_workspace_size(T, H, E, k, F2 // 2, Fs)
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)
    ws[:256] = 0
    return ws


def decode(x, w, k, ws=None, **kw):
    from serve_invariant_moe_gb300 import binding
    ws = space(x.shape[0], w, k) if ws is None else ws
    got = binding.moe_layer_decode(x, w["w_router"], w["w13"], w["w2"], k, ws, w.get("ws13"), w.get("ws2"), **kw)
    binding.check_status(ws)
    assert (ws[192:256] == 0).all()
    return got


def separate(x, w, k, routing=None):
    """The same layer through its separate calls."""
    from serve_invariant_moe_gb300 import binding
    T, H = x.shape
    E, F = w["w13"].shape[0], w["w13"].shape[1] // 2
    Fs = w["ws13"].shape[0] // 2 if "ws13" in w else 0
    ws = binding.new_workspace(binding.workspace_size(T, H, E, k, F, Fs))
    shared = dict(x_shared=x, ws13=w["ws13"], ws2=w["ws2"]) if Fs else {}
    if routing is None:
        r = binding.moe_route_topk(x, w["w_router"], k, ws)
        logits, xp = r["logits"], r["xp"]
    else:
        logits = binding.moe_router_logits(x, w["w_router"], ws)
        r = routing.select(logits, k, ws)
        xp = binding.moe_permute_rows(x, r["plan"], E, k)
    f = binding.moe_grouped_ffn(xp, r["plan"], w["w13"], w["w2"], T, k, ws, **shared)
    bf = torch.empty(T, H, dtype=BF, device=DEV)
    out = binding.moe_combine(f["y"], r["topk_w"], r["plan"], T, H, E, k, y_shared=f["y_shared"], out_bf16=bf)
    binding.check_status(ws)
    return dict(out=out, out_bf16=bf, logits=logits, topk_idx=r["topk_idx"], topk_w=r["topk_w"])


def same(got, want):
    for n in want:
        a, b = got[n], want[n]
        assert torch.equal(a.view(torch.int32 if a.element_size() == 4 else torch.int16),
                           b.view(torch.int32 if b.element_size() == 4 else torch.int16)), n


@pytest.mark.parametrize("E,H,F,Fs,k", [(8, 256, 512, 0, 2), (128, 512, 256, 0, 8), (256, 1024, 384, 256, 8),
                                        (64, 192, 128, 128, 1), (32, 2048, 768, 0, 32), (512, 256, 128, 128, 10)])
@pytest.mark.parametrize("T", [1, 2, 7, 16])
def test_bits_of_the_separate_calls(T, E, H, F, Fs, k):
    w, x = weights(E, H, F, Fs), tokens(T, H)
    same(decode(x, w, k, out_bf16=True), separate(x, w, k))


@pytest.mark.parametrize("score,bias,n_group,topk_group,renorm,scale",
                         [("sigmoid", True, 8, 4, True, 2.5), ("sigmoid", False, 1, 1, False, 1.0), ("softmax", False, 1, 1, True, 1.0),
                          ("softmax", False, 16, 3, False, 2.0), ("sigmoid", True, 1, 1, True, 1.0)])
@pytest.mark.parametrize("E", [64, 160, 320])
def test_bits_of_the_separate_calls_with_scores(E, score, bias, n_group, topk_group, renorm, scale):
    from serve_invariant_moe_gb300 import api
    w, x = weights(E, 384, 128, 128), tokens(5, 384)
    b = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)).to(DEV) if bias else None
    routing = api.Routing(score, b, n_group, topk_group, renorm, scale)
    got = decode(x, w, 6, out_bf16=True, score=score, bias=b, n_group=n_group, topk_group=topk_group, renormalize=renorm,
                 scale=scale)
    same(got, separate(x, w, 6, routing))


def reference(x, w, idx, gates):
    """64 bits on the given choice, with the bound of the module's text."""
    x64 = x.double()
    T, k = idx.shape
    out, bound = 0.0, 0.0

    def expert(rows, w13, w2):
        g, u = (rows @ w13.double().T).chunk(2, -1)
        mag = (rows.abs() @ w13.double().abs().T) * (2 * rows.shape[-1] * 2.0 ** -24)
        dg, du = mag.chunk(2, -1)
        s = torch.sigmoid(g)
        h = (g * s * u)
        dh = 1.2 * dg * u.abs() + (g * s).abs() * du + 2 * 2.0 ** -8 * h.abs()     # |silu'| <= 1.1
        K = h.shape[-1]
        y = h @ w2.double().T
        return y, (dh + 2 * K * 2.0 ** -24 * h.abs()) @ w2.double().abs().T
    out, bound = torch.zeros_like(x64), torch.zeros_like(x64)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            y, b = expert(x64[t:t + 1], w["w13"][e], w["w2"][e])
            out[t] += float(gates[t, j]) * y[0]
            bound[t] += abs(float(gates[t, j])) * (b[0] + (k + 2) * 2.0 ** -24 * y[0].abs())
    if "ws13" in w:
        y, b = expert(x64, w["ws13"], w["ws2"])
        out += y
        bound += b + 2.0 ** -23 * y.abs()
    return out, bound


@pytest.mark.parametrize("T,E,H,F,Fs,k", [(1, 1, 64, 64, 0, 1), (16, 3, 64, 64, 64, 3), (5, 21, 192, 64, 192, 4), (16, 60, 320, 192, 64, 9),
                                          (3, 500, 128, 64, 0, 32), (2, 17, 64, 1024, 0, 2), (4, 5, 4160, 64, 0, 2), (9, 16, 8256, 64, 64, 1)])
def test_odd_sizes_against_64_bits(T, E, H, F, Fs, k):
    w, x = weights(E, H, F, Fs), tokens(T, H)
    got = decode(x, w, k, out_bf16=True)
    l64 = x.double() @ w["w_router"].double().T
    mag = x.double().abs() @ w["w_router"].double().abs().T
    assert ((got["logits"].double() - l64).abs() <= 2 * H * 2.0 ** -24 * mag).all()
    top = torch.sort(got["logits"], dim=-1, descending=True, stable=True)
    assert torch.equal(got["topk_idx"].long(), top.indices[:, :k])
    gates = torch.softmax(top.values[:, :k].double(), -1)
    assert torch.allclose(got["topk_w"].double(), gates, rtol=1e-5, atol=1e-30)
    out, bound = reference(x, w, got["topk_idx"], got["topk_w"])
    assert ((got["out"].double() - out).abs() <= bound + 1e-30).all()
    assert torch.equal(got["out_bf16"], got["out"].to(BF))


@pytest.mark.parametrize("T,E,H,F,Fs,k", [(2, 6, 32768, 64, 64, 2), (3, 4, 128, 9216, 64, 2)])
def test_the_widest_rows(T, E, H, F, Fs, k):
    w, x = weights(E, H, F, Fs), tokens(T, H)
    got = decode(x, w, k)
    out, bound = reference(x, w, got["topk_idx"], got["topk_w"])
    assert ((got["out"].double() - out).abs() <= bound + 1e-30).all()


@pytest.mark.parametrize("score,n_group,topk_group", [(None, 1, 1), ("sigmoid", 32, 9), ("softmax", 4, 4)])
def test_the_most_pairs(score, n_group, topk_group):
    """16 tokens with 32 of 512 experts each."""
    from serve_invariant_moe_gb300 import api
    w, x = weights(512, 256, 128, 128), tokens(16, 256)
    if score is None:
        return same(decode(x, w, 32, out_bf16=True), separate(x, w, 32))
    bias = 0.1 * torch.randn(512, generator=torch.Generator().manual_seed(3)).to(DEV)
    got = decode(x, w, 32, out_bf16=True, score=score, bias=bias, n_group=n_group, topk_group=topk_group)
    same(got, separate(x, w, 32, api.Routing(score, bias, n_group, topk_group, True, 1.0)))


def test_graphs_that_share_a_workspace():
    """Of different layers and sizes, replayed in turn on one stream, with eager calls in between."""
    from serve_invariant_moe_gb300 import binding
    a, b = weights(128, 512, 256, 128), weights(8, 256, 512)
    ws = space(16, a, 8)
    calls = [(a, 8, tokens(16, 512)), (b, 2, tokens(3, 256)), (a, 8, tokens(1, 512, 4))]
    want = [decode(x, w, k)["out"] for w, k, x in calls]

    def run(w, k, x):
        return binding.moe_layer_decode(x, w["w_router"], w["w13"], w["w2"], k, ws, w.get("ws13"), w.get("ws2"))["out"]
    graphs, outs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(*c))
    for i in (0, 1, 2, 1, 0, 0, 2):
        outs[i].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(run(*calls[(i + 1) % 3]), want[(i + 1) % 3])
        assert torch.equal(outs[i], want[i])
    binding.check_status(ws)


def test_tokens_that_choose_alike_and_not():
    """All tokens the same (every expert has 16 rows), and all of different experts."""
    w, x = weights(32, 256, 128, 128), tokens(16, 256)
    x[:] = x[0]
    got = decode(x, w, 4, out_bf16=True)
    same(got, separate(x, w, 4))
    assert (got["out"] == got["out"][0]).all()
    apart = weights(16, 256, 128)
    apart["w_router"] = torch.zeros(16, 256, dtype=BF, device=DEV)
    apart["w_router"][torch.arange(16), torch.arange(16)] = 1.0
    x = tokens(16, 256)
    x[torch.arange(16), torch.arange(16)] = 100.0
    got = decode(x, apart, 1, out_bf16=True)
    assert torch.equal(got["topk_idx"][:, 0].cpu(), torch.arange(16, dtype=torch.int32))
    same(got, separate(x, apart, 1))


def test_a_tokens_bits_are_its_own():
    w, x = weights(64, 512, 256, 128), tokens(16, 512)
    whole = decode(x, w, 8)
    for t in (0, 9, 15):
        same({n: v[t:t + 1] if v is not None else v for n, v in whole.items()},
             {n: v for n, v in decode(x[t:t + 1].contiguous(), w, 8).items() if v is not None})


def test_special_tokens_stay_their_own():
    w, x = weights(64, 256, 128, 128), tokens(6, 256)
    clean = decode(x, w, 4)
    x[1, 3], x[2, 5], x[3] = float("nan"), float("inf"), 0.0
    got = decode(x, w, 4)
    want = separate(x, w, 4)
    same({n: v for n, v in got.items() if n in ("topk_idx",)}, {"topk_idx": want["topk_idx"]})
    for t in (0, 4, 5):
        for n in ("out", "logits", "topk_idx", "topk_w"):
            assert torch.equal(got[n][t], clean[n][t]), (n, t)
    assert torch.isnan(got["out"][1]).all() and (got["out"][3] == 0).all()


def test_outputs_given_and_skipped():
    w, x = weights(8, 256, 128), tokens(3, 256)
    want = decode(x, w, 2, out_bf16=True)
    buf = {n: torch.empty_like(v) for n, v in want.items()}
    got = decode(x, w, 2, **buf)
    for n in buf:
        assert got[n].data_ptr() == buf[n].data_ptr()
    same(got, want)
    assert decode(x, w, 2)["out_bf16"] is None
    assert decode(x, w, 2, out=False, out_bf16=True)["out"] is None
    assert decode(x[:0], w, 2)["out"].shape == (0, 256)


def test_many_calls_on_one_workspace():
    """Different sizes in turn, nothing cleared between them; the counters are the workspace's first 256 bytes' again."""
    from serve_invariant_moe_gb300 import binding
    a, b = weights(128, 512, 256, 128), weights(8, 256, 512)
    xs = [tokens(T, 512, T) for T in (1, 16, 5)], [tokens(T, 256, T) for T in (2, 13)]
    ws = space(16, a, 8)
    want = [decode(x, a, 8)["out"] for x in xs[0]], [decode(x, b, 2)["out"] for x in xs[1]]
    for _ in range(40):
        for w, k, x, o in [(a, 8, x, o) for x, o in zip(xs[0], want[0])] + [(b, 2, x, o) for x, o in zip(xs[1], want[1])]:
            got = binding.moe_layer_decode(x, w["w_router"], w["w13"], w["w2"], k, ws, w.get("ws13"), w.get("ws2"))
            assert torch.equal(got["out"], o)
    binding.check_status(ws)


def test_streams_and_a_captured_call():
    from serve_invariant_moe_gb300 import binding
    w = weights(128, 512, 256, 128)
    xs = [tokens(4, 512, s) for s in range(4)]
    want = [decode(x, w, 8)["out"] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [space(4, w, 8) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(60):                              # two streams, a workspace each
        with torch.cuda.stream(streams[i % 2]):
            outs.append((i % 4, binding.moe_layer_decode(xs[i % 4], w["w_router"], w["w13"], w["w2"], 8, spaces[i % 2],
                                                         w["ws13"], w["ws2"])["out"]))
    torch.cuda.synchronize()
    for i, o in outs:
        assert torch.equal(o, want[i])
    ws, x = space(4, w, 8), xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.moe_layer_decode(x, w["w_router"], w["w13"], w["w2"], 8, ws, w["ws13"], w["ws2"])["out"]
    for i in (3, 1, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    for s in (ws, *spaces):
        binding.check_status(s)


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    w, x = weights(8, 256, 128), tokens(3, 256)
    ws = space(16, w, 2)
    f = lambda **k: binding.moe_layer_decode(**{**dict(x=x, w_router=w["w_router"], w13=w["w13"], w2=w["w2"], k=2, workspace=ws), **k})   # noqa: E731
    f()
    with pytest.raises(InvmoeError, match="T=17"):
        f(x=tokens(17, 256))
    with pytest.raises(InvmoeError, match="k=9"):
        f(k=9)
    with pytest.raises(InvmoeError, match="need a score"):
        f(scale=2.0)
    with pytest.raises(InvmoeError, match="workspace"):
        f(workspace=ws[:4096].clone())
    with pytest.raises(InvmoeError, match="both NULL"):
        f(out=False)
    with pytest.raises(ValueError, match="score"):
        f(score="relu")
    with pytest.raises(InvmoeError, match="groups"):
        f(score="sigmoid", n_group=4, topk_group=1, k=3)
    with pytest.raises(InvmoeError, match="overlaps"):
        f(out=False, out_bf16=x)
    with pytest.raises(ValueError, match="w2"):
        f(w2=w["w2"].float())


def test_an_error_that_was_reported_leaves_a_clear_workspace():
    """Counters that calls on one workspace at once, or a call given up, have left behind go with the status."""
    from serve_invariant_moe_gb300 import binding
    w, x = weights(8, 256, 128), tokens(4, 256)
    want = decode(x, w, 2, out_bf16=True)
    ws = space(4, w, 2)
    ws[:256] = 3
    ws[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError):
        binding.check_status(ws)
    assert not ws[:256].any()
    same(decode(x, w, 2, ws, out_bf16=True), want)
