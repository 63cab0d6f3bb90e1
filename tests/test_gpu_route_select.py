"""Expert choice by scores on the GPU against a plain 64-bit reference, and its backward against the formula's gradient.

The choice is compared exactly: tokens whose 64-bit choice values come within 1e-5 of each other without being equal are
left out of the inputs (fp32 scores are within 4e-7), ties are made on purpose.  Weights: a score has relative error
below 8 * 2^-24 (exp, sum, division), renormalising adds k + 2 roundings: 5e-6 relative covers k <= 32.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def scores64(l, kind):
    with np.errstate(all="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.exp(l - np.where(m == -np.inf, 0, m))
        s = e.sum(1, keepdims=True)
        return np.where(s == 0, 0.0, e / s)


def order(v):
    """Indices by value, largest first, ties to the lower index, NaN last."""
    v = np.asarray(v, np.float64) + 0.0
    return sorted(range(len(v)), key=lambda i: (np.isnan(v[i]), -v[i] if not np.isnan(v[i]) else 0.0, i))


def reference(l, k, kind, bias, groups, kept, renorm, scale):
    l = l.double().numpy()
    T, E = l.shape
    p = scores64(l, kind)
    c = l if bias is None else p + bias.double().numpy()
    per = E // groups
    idx, gap = np.zeros((T, k), np.int64), np.full(T, np.inf)
    for t in range(T):
        live = np.ones(E, bool)
        if kept < groups:
            value = []
            for g in range(groups):
                top = c[t, g * per:(g + 1) * per][order(c[t, g * per:(g + 1) * per])]
                value.append(top[0] if bias is None or per == 1 else top[0] + top[1])
            o = order(value)
            gap[t] = min(gap[t], near(value[o[kept - 1]], value[o[kept]]))
            for g in o[kept:]:
                live[g * per:(g + 1) * per] = False
        o = [e for e in order(c[t]) if live[e]]
        idx[t] = o[:k]
        for j in range(min(k, len(o) - 1)):
            gap[t] = min(gap[t], near(c[t, o[j]], c[t, o[j + 1]]))
    w = np.take_along_axis(p, idx, 1)
    if renorm:
        s = w.sum(1, keepdims=True)
        with np.errstate(all="ignore"):
            w = np.where(s == 0, 0.0, w / s)
    return idx, scale * w, gap


def near(a, b):
    """How far two decided values are apart; equal ones (a tie, decided by index) and special ones do not count."""
    if a == b or not np.isfinite(a) or not np.isfinite(b):
        return np.inf
    return abs(a - b)


CASES = [(1, 8, 1, 1, 1), (5, 60, 4, 1, 1), (40, 128, 8, 1, 1), (33, 256, 8, 8, 4), (70, 160, 6, 8, 3), (20, 64, 4, 4, 1),
         (9, 21, 5, 3, 2), (300, 256, 8, 1, 1), (17, 512, 32, 16, 8), (4, 1024, 16, 32, 5), (6, 1000, 12, 1, 1),
         (8, 32, 16, 32, 20), (3, 1, 1, 1, 1), (11, 96, 3, 2, 1)]


@pytest.mark.parametrize("score,with_bias", [("sigmoid", True), ("sigmoid", False), ("softmax", False), ("softmax", True)])
@pytest.mark.parametrize("T,E,k,groups,kept", CASES)
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0)])
def test_select(T, E, k, groups, kept, score, with_bias, renorm, scale):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T + E + k)
    l = torch.randn(T, E, generator=g) * 1.5
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    idx, w, gap = reference(l, k, score, bias, groups, kept, renorm, scale)
    r = binding.moe_route_select(l.to(DEV), k, score, None if bias is None else bias.to(DEV), groups, kept, renorm, scale)
    ok = gap > 1e-5
    assert ok.mean() > 0.3
    assert np.array_equal(r["topk_idx"].cpu().numpy()[ok], idx[ok])
    assert np.allclose(r["topk_w"].double().cpu().numpy()[ok], w[ok], rtol=5e-6, atol=1e-30)


@pytest.mark.parametrize("score,with_bias", [("sigmoid", True), ("softmax", False)])
@pytest.mark.parametrize("T,E,k,groups,kept", [(20, 256, 8, 4, 2), (9, 1024, 8, 4, 3), (12, 192, 6, 3, 1), (7, 320, 5, 5, 2)])
def test_select_with_groups_of_several_warps_widths(T, E, k, groups, kept, score, with_bias):
    test_select(T, E, k, groups, kept, score, with_bias, True, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_ties_go_to_the_lower_index(score, groups, kept):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(1)
    # many equal logits, -0 and +0 among them; no two different pairs of scores have nearly equal sums
    l = torch.tensor([-2.0, 0.0, 1.0])[torch.randint(0, 3, (200, 32), generator=g)]
    l[::3] *= -1.0
    bias = torch.full((32,), 0.125)
    for b in (None, bias):
        idx, w, _ = reference(l, 6, score, b, groups, kept, True, 1.0)
        r = binding.moe_route_select(l.to(DEV), 6, score, None if b is None else b.to(DEV), groups, kept)
        assert np.array_equal(r["topk_idx"].cpu().numpy(), idx)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_and_special_rows(score, renorm):
    from serve_invariant_moe_gb300 import binding
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    l = torch.randn(6, 16, generator=torch.Generator().manual_seed(2))
    l[0] = -inf                       # nothing left
    l[1, 1:] = -inf                   # one expert left
    l[2, 3:] = low                    # masked with the lowest value
    l[3, 5] = nan
    l[4] = low
    r = binding.moe_route_select(l.to(DEV), 4, score, renormalize=renorm)
    idx, w = r["topk_idx"].cpu(), r["topk_w"].cpu()
    assert idx[0].tolist() == [0, 1, 2, 3] and (w[0] == 0).all()
    assert idx[1].tolist() == [0, 1, 2, 3] and (w[1, 1:] == 0).all() and w[1, 0] > 0
    assert sorted(idx[2, :3].tolist()) == [0, 1, 2] and idx[2, 3] == 3 and w[2, 3] == 0 and torch.isfinite(w[2]).all()
    assert 5 not in idx[3].tolist()
    assert torch.isnan(w[3]).all() if score == "softmax" else torch.isfinite(w[3]).all()
    assert idx[4].tolist() == [0, 1, 2, 3]
    assert (w[4] == 0).all() if score == "sigmoid" else torch.allclose(w[4], torch.full((4,), 0.25 if renorm else 1 / 16))
    want = binding.moe_route_select(l[5:].to(DEV), 4, score, renormalize=renorm)
    assert torch.equal(want["topk_w"], r["topk_w"][5:]) and torch.equal(want["topk_idx"], r["topk_idx"][5:])
    # a NaN is taken when nothing else is left
    m = torch.full((1, 8), nan)
    m[0, 6] = 1.0
    assert binding.moe_route_select(m.to(DEV), 3, "sigmoid")["topk_idx"][0].tolist() == [6, 0, 1]


def test_the_softmax_sum_does_not_depend_on_the_order():
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(3)
    l = torch.randn(64, 200, generator=g) * 4
    perm = torch.randperm(200, generator=g)
    a = binding.moe_route_select(l.to(DEV), 8, "softmax", renormalize=False)
    b = binding.moe_route_select(l[:, perm].contiguous().to(DEV), 8, "softmax", renormalize=False)
    assert torch.equal(a["topk_w"], b["topk_w"])
    assert torch.equal(a["topk_idx"].cpu().long(), perm[b["topk_idx"].cpu().long()])


@pytest.mark.parametrize("T", [0, 1, 5, 64, 300, 1000])
def test_plan_and_batch(T):
    """The plan is moe_route_topk's counting sort; a token's bits do not depend on its batch."""
    from oracle import moe as omoe
    from serve_invariant_moe_gb300 import binding
    E, k = 24, 3
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(DEV)
    bias = torch.linspace(-0.1, 0.1, E, device=DEV)
    ws = binding.new_workspace(binding.workspace_size(T, 64, E, k))
    r = binding.moe_route_select(l, k, bias=bias, plan=True, workspace=ws)
    plan = r["plan"].cpu().numpy()
    if T == 0:
        assert (plan[:2 * E + 1] == 0).all()
        return
    ref = omoe.dispatch_plan(r["topk_idx"].cpu().numpy(), E)
    S = T * k
    parts = [plan[:E], plan[E:2 * E + 1], plan[2 * E + 1:2 * E + 1 + S], plan[2 * E + 1 + S:2 * E + 1 + 2 * S].reshape(T, k)]
    for got, want in zip(parts, ref):
        assert np.array_equal(got, want)
    one = binding.moe_route_select(l[T // 2:T // 2 + 1].contiguous(), k, bias=bias)
    assert torch.equal(one["topk_w"], r["topk_w"][T // 2:T // 2 + 1])


def grad64(l, idx, dw, score, renorm, scale):
    l = l.double().requires_grad_()
    p = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    w = p.gather(1, idx.long())
    w = scale * (w / w.sum(1, keepdim=True) if renorm else w)
    (w * dw.double()).sum().backward()
    return l.grad.numpy()


def test_the_gradient_against_differences():
    """The 64-bit gradient the kernel is compared with, by central differences of the weights' formula."""
    g = torch.Generator().manual_seed(4)
    l, dw = torch.randn(2, 6, generator=g), torch.randn(2, 3, generator=g)
    idx = torch.tensor([[4, 0, 2], [1, 5, 3]])
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            d = grad64(l, idx, dw, score, renorm, 2.5)

            def f(x):
                p = torch.from_numpy(scores64(x.numpy(), score)).gather(1, idx)
                return float((2.5 * (p / p.sum(1, keepdim=True) if renorm else p) * dw.double()).sum())
            for t in range(2):
                for e in range(6):
                    h = torch.zeros(2, 6, dtype=torch.float64)
                    h[t, e] = 1e-6
                    assert abs((f(l.double() + h) - f(l.double() - h)) / 2e-6 - d[t, e]) < 1e-7


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (False, 1.0)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (5, 60, 4), (40, 256, 8), (300, 128, 8), (3, 1024, 32), (7, 1, 1), (9, 21, 5)])
def test_select_backward(T, E, k, score, renorm, scale):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T + E)
    l = torch.randn(T, E, generator=g) * 1.5
    dw = torch.randn(T, k, generator=g)
    idx = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    b16 = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, renorm, scale, dlogits_bf16=b16)
    ref = grad64(l, idx, dw, score, renorm, scale)
    # one fp32 rounding of each factor and a k-term sum, relative to the terms before they cancel
    p = scores64(l.double().numpy(), score)
    w = np.take_along_axis(p, idx.numpy().astype(np.int64), 1)
    d = np.abs(scale * dw.double().numpy())
    s = w.sum(1, keepdims=True) if renorm else 1.0
    size = ((d + (d * w).sum(1, keepdims=True) / s) / s).max(1, keepdims=True) * np.maximum(p, 0)
    tol = (40 + k) * 2.0 ** -24 * size + 1e-30
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    assert torch.equal(b16, got.to(torch.bfloat16))
    only = torch.empty_like(b16)
    assert binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, renorm, scale, dlogits=False,
                                             dlogits_bf16=only) is None
    assert torch.equal(only, b16)


def test_backward_of_masked_rows_and_bad_indices():
    from serve_invariant_moe_gb300 import binding
    l = torch.randn(3, 8, generator=torch.Generator().manual_seed(5))
    l[0] = -float("inf")
    idx = torch.tensor([[0, 1], [2, 99], [-1, 3]], dtype=torch.int32)
    dw = torch.ones(3, 2)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            d = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, renorm).cpu()
            assert (d[0] == 0).all() and torch.isfinite(d).all()
            one = binding.moe_route_select_backward(l[1:2].to(DEV), idx[1:2, :1].contiguous().to(DEV),
                                                    dw[1:2, :1].contiguous().to(DEV), score, renorm).cpu()
            assert torch.equal(d[1:2], one)


@pytest.mark.parametrize("score,renorm", [("sigmoid", False), ("softmax", False), ("softmax", True)])
def test_backward_of_an_expert_chosen_twice(score, renorm):
    """Its entry is the sum of both gradients.  With equal dw the renormalised ones are 0 up to rounding, the others
    dw (2 ds/dl): the bound is 16 roundings of the sum of the absolute terms, which are at most 2."""
    from serve_invariant_moe_gb300 import binding
    l = torch.randn(5, 40, generator=torch.Generator().manual_seed(6))
    idx = torch.tensor([[3, 3], [0, 39], [33, 33], [7, 8], [1, 1]], dtype=torch.int32)
    dw = torch.ones(5, 2)
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, renorm).double().cpu()
    x = l.double().requires_grad_(True)
    sc = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = sc.gather(1, idx.long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    w.sum().backward()
    assert (got - x.grad).abs().max() <= 16 * 2 * 2.0 ** -24


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    l = torch.zeros(4, 24, device=DEV)
    for args in [dict(score="relu"), dict(bias=torch.zeros(23, device=DEV)), dict(bias=torch.zeros(24)),
                 dict(topk_idx=torch.zeros(4, 2, dtype=torch.int64, device=DEV)), dict(plan=True)]:
        with pytest.raises(ValueError):
            binding.moe_route_select(l, 2, **args)
    with pytest.raises(ValueError):
        binding.moe_route_select(l.double(), 2)
    with pytest.raises(ValueError):
        binding.moe_route_select(l.t(), 2)
    for k, args, code in [(25, {}, -1), (33, {}, -2), (2, dict(n_group=5), -1), (2, dict(n_group=4, topk_group=5), -1),
                          (7, dict(n_group=4, topk_group=1), -1), (0, {}, -1)]:
        with pytest.raises(InvmoeError) as e:
            binding.moe_route_select(l, k, **args)
        assert e.value.code == code
    with pytest.raises(InvmoeError) as e:
        binding.moe_route_select(torch.zeros(1, 1040, device=DEV), 2)
    assert e.value.code == -2
    with pytest.raises(InvmoeError) as e:
        binding.moe_route_select(l, 2, plan=True, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == -3
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        binding.moe_route_select_backward(l, idx, torch.zeros(4, 3, device=DEV))
    with pytest.raises(InvmoeError) as e:
        binding.moe_route_select_backward(l, idx, torch.zeros(4, 2, device=DEV), dlogits=False)
    assert e.value.code == -1
