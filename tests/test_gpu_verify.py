"""Verification of drafted tokens on the GPU against a request-by-request oracle in 64 bits.

Tolerance.  exp((z - m) / tau) in fp32: three roundings (the difference, log2(e) / tau, their product) of an argument of at most
104 (beyond it the weight is 0 in fp32) move it by 3 * 104 * 2^-24, the exponential adds 2^-22, the reciprocals of the sum and of
the noise 2^-22 each, and a sum of at most 32 + 13 + (V / 8192 / 32 + 5) terms in a row 60 * 2^-24: REL = 4e-5 of a probability
covers it.  A decision has to be the oracle's except where its two
sides are within that of one another, and a drawn token's score has to be within that of the largest.  The logarithm of a
probability is within REL + 2^-23 of its value.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 4e-5
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def make(B, D, V, dtype=F32, draft=True, ragged=False, tau=1.0, spread=2.5, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * B + 10 * D + V)
    z = spread * torch.randn(B, D + 1, V, generator=g)
    a = dict(logits=z.to(dtype), noise=torch.empty(B, V).exponential_(generator=g), temperature=tau)
    if D:
        near = z[:, :D] + 0.5 * torch.randn(B, D, V, generator=g)
        a["draft_tokens"] = (near - torch.empty(B, D, V).exponential_(generator=g).log()).argmax(-1).to(torch.int32)
        a["accept_u"] = torch.rand(B, D, generator=g)
        if draft:
            a["draft_logits"] = near.to(dtype)
        if ragged:
            a["n_draft"] = torch.randint(0, D + 1, (B,), generator=g).to(torch.int32)
    return a


def call(a, workspace=None):
    from serve_invariant_moe_gb300 import binding
    B, rows, V = a["logits"].shape
    if workspace is None:       # any content
        workspace = torch.randint(0, 256, (binding.verify_workspace_size(B, rows - 1, V),), dtype=torch.uint8, device=DEV)
    a = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    got = binding.verify_drafts(a.pop("logits"), a.pop("noise"), workspace, **a)
    return {n: t.cpu().numpy() for n, t in got.items()}


def usable(t):
    z = t.double().numpy()
    return np.where(np.isnan(z), -np.inf, np.minimum(z, np.finfo(np.float32).max))


def probabilities(z, tau):
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z), np.full_like(z, -np.inf)
    x = np.where(z == -np.inf, -np.inf, (z - m) / tau)
    e = np.exp(x)
    return e / e.sum(), x - math.log(e.sum())


def check(got, a):
    B, rows, V = a["logits"].shape
    D = rows - 1
    assert got["tokens"].shape == (B, D + 1) and got["n_accepted"].shape == (B,) and got["logp"].shape == (B, D + 1)
    for b in range(B):
        t = a["temperature"]
        tau = float(t[b]) if isinstance(t, torch.Tensor) else float(t)
        greedy = not tau > 0
        tau = 1.0 if greedy else tau
        n_draft = int(a["n_draft"][b]) if "n_draft" in a else D
        n = int(got["n_accepted"][b])
        assert 0 <= n <= n_draft
        z = usable(a["logits"][b])
        for i in range(n + 1):
            p, lp = probabilities(z[i], tau)
            token = int(got["tokens"][b, i])
            if i < n_draft:
                x = int(a["draft_tokens"][b, i])
                inside = 0 <= x < V
                px = p[x] if inside else 0.0
                if "draft_logits" in a:
                    q, _ = probabilities(usable(a["draft_logits"][b, i]), tau)
                    qx = q[x] if inside else 0.0
                else:
                    q = np.zeros(V)
                    qx = 1.0
                    if inside:
                        q[x] = 1.0
                if greedy:
                    ok = inside and p.max() > 0 and x == int(np.flatnonzero(z[i] == z[i].max())[0])
                    assert ok == (i < n), (b, i)
                else:
                    uq = float(a["accept_u"][b, i]) * qx
                    ok = uq < px
                    if ok != (i < n):
                        assert abs(uq - px) <= 2 * REL * max(uq, px), (b, i, uq, px)
                if i < n:
                    assert token == x
            if i == n:
                if z[i].max() == -np.inf:
                    assert token == -1 and got["logp"][b, i] == -np.inf
                    continue
                if greedy:
                    assert token == int(np.flatnonzero(z[i] == z[i].max())[0])
                else:
                    e = a["noise"][b].double().numpy()
                    w, err = p, REL * p
                    if i < n_draft:
                        left = np.maximum(p - q, 0.0)
                        if (left > 0).any():
                            w, err = left, REL * (p + q)
                    with np.errstate(divide="ignore", invalid="ignore"):
                        score, slack = w / e, err / e
                    score = np.where((w > 0) & (score >= 0), score, -1.0)
                    assert 0 <= token < V
                    slack = np.where(np.isfinite(slack), slack, 0.0)
                    if np.isinf(score.max()):
                        assert token == int(np.flatnonzero(np.isinf(score))[0])
                    else:
                        assert score[token] + slack[token] >= (score - slack).max() and w[token] + err[token] > 0
            assert abs(got["logp"][b, i] - lp[token]) <= REL + 2.0 ** -23 * abs(lp[token]) + abs(lp[token]) * 2.0 ** -22
        assert (got["tokens"][b, n + 1:] == -1).all() and (got["logp"][b, n + 1:] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("D", [0, 1, 4, 32])
@pytest.mark.parametrize("V", [1, 2, 7, 100, 2051, 8192, 8193, 20012])
def test_against_the_oracle(V, D, draft, dtype):
    a = make(3, D, V, dtype, draft)
    check(call(a), a)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [151552, 151557])
def test_a_large_vocabulary(V, dtype):
    a = make(2, 3, V, dtype, ragged=True, tau=torch.tensor([0.7, 1.3]))
    check(call(a), a)


@pytest.mark.parametrize("V", [500, 9000])
def test_ragged_drafts_and_temperatures(V):
    tau = torch.tensor([1.0, 0.0, 0.3, 2.0, 0.0, 1e-6, -1.0, float("nan"), 0.8, 1.0, 1e30, 1e-40])
    a = make(12, 5, V, ragged=True, tau=tau)
    a["n_draft"][:4] = torch.tensor([0, 5, 9, -3], dtype=torch.int32)     # clamped to [0, D]
    for b in (1, 4, 6, 7):                                               # a greedy drafter that is often right
        a["draft_tokens"][b] = a["logits"][b, :5].argmax(-1).to(torch.int32)
    a["draft_tokens"][4, 2] += 1
    got = call(a)
    a["n_draft"].clamp_(0, 5)
    check(got, a)
    assert got["n_accepted"][4] == min(2, int(a["n_draft"][4]))


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("D", [0, 2])
def test_an_infinite_temperature(D, own):
    """Every logit but -inf has the same probability, also where a chunk has none and behind the end of a row."""
    a = make(3, D, 20012, tau=torch.full((3,), math.inf) if own else math.inf)
    a["logits"][:, :, 100:17000] = -math.inf
    if D:
        a["draft_logits"][1:, :, 5:15000] = -math.inf
        a["draft_tokens"][0, 0] = 7
    got = call(a)
    check(got, a)
    assert np.allclose(got["logp"][got["tokens"] >= 0], -math.log(20012 - 16900), rtol=0, atol=REL + 8 * 2.0 ** -22)


def test_scalar_temperatures():
    for tau in (0.0, 0.5, 3.0):
        a = make(4, 3, 300, tau=tau)
        check(call(a), a)


def test_the_drafter_that_is_the_target_is_always_right():
    a = make(6, 8, 5000)
    a["draft_logits"] = a["logits"][:, :8].clone()
    a["accept_u"].fill_(1 - 2.0 ** -24)
    got = call(a)
    assert (got["n_accepted"] == 8).all()
    check(got, a)


def test_a_rejection_that_leaves_nothing_draws_from_the_target():
    """p = q in every bit, but the draft token lies outside the vocabulary: max(p - q, 0) is zero everywhere."""
    a = make(4, 1, 3000)
    a["draft_logits"] = a["logits"][:, :1].clone()
    a["draft_tokens"][:] = torch.tensor([[-1], [3000], [2 ** 31 - 1], [-2 ** 31]], dtype=torch.int32)
    got = call(a)
    assert (got["n_accepted"] == 0).all()
    check(got, a)


@pytest.mark.parametrize("D", [0, 2])
def test_masked_logits(D):
    """-inf and NaN are no tokens, +inf takes all the mass, a row of neither draws nothing; a mask of the type's lowest value
    is a logit like any other."""
    V = 8200
    a = make(8, D, V, draft=False)
    z = a["logits"]
    z[0] = float("-inf")
    z[0, :, 8195] = -3.0
    z[1] = float("nan")
    z[1, :, 17] = 1.0
    z[2] = float("-inf")
    z[3, :, 4000] = float("inf")
    z[4] = torch.finfo(F32).min
    z[5, :, ::2] = float("-inf")
    z[6, :, :8192] = float("-inf")
    if D:
        a["draft_tokens"][0] = 8195
        a["draft_tokens"][1] = 16
        a["draft_tokens"][3] = 4000
        a["draft_tokens"][5] = 2
    got = call(a)
    check(got, a)
    assert got["tokens"][0, got["n_accepted"][0]] == 8195 and got["tokens"][2, 0] == -1 and got["tokens"][1, 0] == 17


def test_masked_drafters():
    a = make(4, 2, 1000)
    a["draft_logits"][0] = float("-inf")
    a["draft_logits"][1] = float("nan")
    a["draft_logits"][2, :, 500:] = float("-inf")
    check(call(a), a)


def test_equal_scores_and_odd_noise():
    """Equal scores go to the lower index; a noise of 0 wins, negative or NaN noise never does, infinite noise comes last."""
    V = 20000
    a = make(6, 0, V)
    a["logits"][:] = 0.5
    a["noise"][:] = 1.0
    a["noise"][1, 12345] = 0.0
    a["noise"][1, 77] = -1.0
    a["noise"][2, :] = float("nan")
    a["noise"][2, 19999] = 3.0
    a["noise"][3, :] = float("inf")
    a["noise"][4, :9000] = 2.0
    a["noise"][5, 3] = -0.0
    assert call(a)["tokens"][:, 0].tolist() == [0, 12345, 19999, 0, 9000, 0]


def test_greedy_ties_go_to_the_lower_index():
    a = make(3, 1, 17000, tau=0.0)
    a["logits"][:] = 0.0
    a["logits"][1, :, [9000, 8191, 16999]] = 4.0
    a["logits"][2, :, [8192, 16000]] = 2.0
    a["draft_tokens"][:] = torch.tensor([[0], [9000], [8192]], dtype=torch.int32)
    got = call(a)
    assert got["n_accepted"].tolist() == [1, 0, 1]
    assert got["tokens"].tolist() == [[0, 0], [8191, -1], [8192, 8192]]
    check(got, a)


def test_a_requests_bits_are_its_own():
    a = make(40, 4, 9001, ragged=True, tau=torch.linspace(0.0, 1.5, 40))
    whole = call(a)
    for b in (0, 7, 39):
        one = {n: t[b:b + 1] if isinstance(t, torch.Tensor) else t for n, t in a.items()}
        alone = call(one)
        for name in whole:
            assert np.array_equal(whole[name][b:b + 1], alone[name]), (b, name)


def test_emitted_tokens_have_the_targets_distribution():
    """60000 requests with the same two rows: the first token's frequencies, accepted or drawn, are p within 5 sigma."""
    B, V = 60000, 12
    g = torch.Generator(device=DEV).manual_seed(3)
    z, zq = torch.randn(V, generator=g, device=DEV), torch.randn(V, generator=g, device=DEV)
    q = torch.softmax(zq, 0)
    drafts = (q / torch.empty(B, V, device=DEV).exponential_(generator=g)).argmax(-1, keepdim=True).to(torch.int32)
    a = dict(logits=z.expand(B, 2, V).contiguous(), noise=torch.empty(B, V, device=DEV).exponential_(generator=g),
             draft_tokens=drafts, draft_logits=zq.expand(B, 1, V).contiguous(), accept_u=torch.rand(B, 1, generator=g, device=DEV),
             temperature=1.0)
    got = call(a)
    p = torch.softmax(z.double(), 0).cpu().numpy()
    seen = np.bincount(got["tokens"][:, 0], minlength=V) / B
    assert (np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / B)).all()
    assert 0.2 < got["n_accepted"].mean() < 0.95
    second = got["tokens"][got["n_accepted"] == 1, 1]
    seen = np.bincount(second, minlength=V) / len(second)
    assert (np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / len(second))).all()


def test_no_requests():
    a = make(0, 2, 50)
    got = call(a)
    assert got["tokens"].shape == (0, 3)


def test_offsets_past_2_31():
    """The last of 15000 requests lies behind 2^31 elements; it gives the bits that it gives alone."""
    B, V = 15000, 151552
    g = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.zeros(B, 1, V, dtype=BF, device=DEV)
    logits[-1].normal_(generator=g)
    noise = torch.ones(B, V, device=DEV)
    noise[-1].exponential_(generator=g)
    whole = call(dict(logits=logits, noise=noise, temperature=1.0))
    alone = call(dict(logits=logits[-1:].clone(), noise=noise[-1:].clone(), temperature=1.0))
    assert (whole["tokens"][:-1] == 0).all()
    for name in whole:
        assert np.array_equal(whole[name][-1:], alone[name])


def test_a_captured_call_replays_with_other_inputs():
    from serve_invariant_moe_gb300 import binding
    a = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in make(5, 3, 9000, ragged=True).items()}
    ws = binding.new_workspace(binding.verify_workspace_size(5, 3, 9000))
    run = lambda: binding.verify_drafts(workspace=ws, **a)   # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (1, 2, 3):
        host = make(5, 3, 9000, ragged=True, seed=seed)
        for n, t in host.items():
            if isinstance(t, torch.Tensor):
                a[n].copy_(t)
        graph.replay()
        got = {n: t.cpu().numpy() for n, t in outs.items()}
        check(got, host)


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    a = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in make(2, 3, 100).items()}
    ws = binding.new_workspace(binding.verify_workspace_size(2, 3, 100))
    ok = lambda **k: binding.verify_drafts(**{**a, "workspace": ws, **k})   # noqa: E731
    ok()
    with pytest.raises(InvmoeError, match="temperature"):
        ok(temperature=-1.0)
    with pytest.raises(InvmoeError, match="temperature"):
        ok(temperature=float("nan"))
    with pytest.raises(InvmoeError, match="workspace"):
        ok(workspace=ws[:256].clone())
    with pytest.raises(ValueError, match="draft_tokens"):
        ok(draft_tokens=None)
    with pytest.raises(ValueError, match="accept_u"):
        ok(accept_u=a["accept_u"].double())
    with pytest.raises(ValueError, match="draft_logits"):
        ok(draft_logits=a["draft_logits"].to(BF))
    with pytest.raises(ValueError, match="noise"):
        ok(noise=a["noise"][:, :99])
    with pytest.raises(ValueError, match="room for drafts"):
        binding.verify_drafts(a["logits"][:, :1].contiguous(), a["noise"], ws, draft_tokens=a["draft_tokens"])
    with pytest.raises(InvmoeError, match="D=33"):
        binding.verify_drafts(torch.zeros(1, 34, 8, device=DEV), torch.ones(1, 8, device=DEV), binding.new_workspace(1 << 20),
                              draft_tokens=torch.zeros(1, 33, dtype=torch.int32, device=DEV),
                              accept_u=torch.zeros(1, 33, device=DEV))
