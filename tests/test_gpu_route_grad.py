"""Gradient of scored routing where scores are near 0 or 1, relative to each entry instead of to its row.

The reference is the gradient in a form without cancellation, in 64 bits, which a CPU test compares with the formula's
automatic gradient.  Tolerances, u = 2^-24: a score has exp's 4 u, two roundings and (softmax) the argument's, u times the
largest difference of two logits; weights add k + 1, a sum over the chosen 2 k, one over the others E / 32 + 5, products 6.
At most two scores and a sum of scores meet in an entry: (64 + 6 k + E / 32 + 3 spread) u covers it, relative to the entry
with every difference taken absolute.
"""
import numpy as np
import pytest
import torch

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def gradient(l, idx, dw, score, renorm, scale):
    """(gradient, the same with every difference absolute), no chosen expert twice."""
    l, dw = l.double().numpy(), dw.double().numpy()
    idx = idx.long().numpy()
    chosen = np.zeros_like(l, bool)
    np.put_along_axis(chosen, idx, True, 1)
    diff = dw[:, :, None] - dw[:, None, :]                    # [t, j, i] = dw_j - dw_i
    if score == "sigmoid":
        e = np.exp(-np.abs(l))
        p, comp = np.where(l >= 0, 1, e) / (1 + e), np.where(l >= 0, e, 1) / (1 + e)
    else:
        e = np.exp(l - l.max(1, keepdims=True))
        p, comp = e / e.sum(1, keepdims=True), np.ones_like(l)
    s, c = np.take_along_axis(p, idx, 1), np.take_along_axis(comp, idx, 1)
    out, size = np.zeros_like(l), np.zeros_like(l)
    if renorm:
        w = s / s.sum(1, keepdims=True)
        own, ab = w * c * (diff * w[:, None, :]).sum(2), w * c * (np.abs(diff) * w[:, None, :]).sum(2)
    elif score == "sigmoid":
        own = dw * s * c
        ab = np.abs(own)
    else:
        rest = np.where(chosen, 0, p).sum(1, keepdims=True)
        own = s * ((diff * s[:, None, :]).sum(2) + dw * rest)
        ab = s * ((np.abs(diff) * s[:, None, :]).sum(2) + np.abs(dw) * rest)
        out = -p * (dw * s).sum(1, keepdims=True)
        size = p * np.abs(dw * s).sum(1, keepdims=True)
    np.put_along_axis(out, idx, own, 1)
    np.put_along_axis(size, idx, ab, 1)
    return scale * out, scale * size


def automatic(l, idx, dw, score, renorm, scale):
    x = l.double().requires_grad_()
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = p.gather(1, idx.long())
    (scale * (w / w.sum(1, keepdim=True) if renorm else w) * dw.double()).sum().backward()
    return x.grad.numpy()


def confident(T, E, k, z, seed):
    """Rows whose first choice lies z above every other expert."""
    g = torch.Generator().manual_seed(seed + E + k)
    l = torch.randn(T, E, generator=g) * 1.5
    idx = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32)
    l[torch.arange(T), idx[:, 0].long()] = l.abs().amax(1) + z
    return l, idx, torch.randn(T, k, generator=g)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_the_reference_is_the_gradient(score, renorm):
    for z in (-2.0, 0.0, 3.0):
        args = confident(6, 9, 3, z, 1)
        ref, size = gradient(*args, score, renorm, 2.5)
        assert (np.abs(ref - automatic(*args, score, renorm, 2.5)) <= 1e-13 * size.max(1, keepdims=True)).all()
        assert (np.abs(ref) <= size * (1 + 1e-12)).all()


SIZES = [(3, 8, 2), (40, 60, 4), (9, 256, 8), (5, 1024, 32), (4, 21, 21)]
GAPS = [0.0, 10.0, 14.0, 18.0, 30.0]


def check(l, idx, dw, score, renorm, scale=2.5):
    from serve_invariant_moe_gb300 import binding
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, renorm, scale)
    ref, size = gradient(l, idx, dw, score, renorm, scale)
    T, E = l.shape
    k = idx.shape[1]
    spread = float((l.amax(1) - l.amin(1)).max()) if score == "softmax" else 0.0
    tol = (64 + 6 * k + E / 32 + 3 * spread) * 2.0 ** -24 * size + 1e-37
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"error / bound {np.max(err / tol):.3g}"


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("z", GAPS)
def test_sigmoid(T, E, k, z):
    check(*confident(T, E, k, z, 2), "sigmoid", False)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("z", GAPS)
def test_renormalised(T, E, k, z, score):
    check(*confident(T, E, k, z, 3), score, True)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_renormalised_over_one_expert_is_constant(score):
    from serve_invariant_moe_gb300 import binding
    l, idx, dw = confident(50, 40, 1, 0.0, 4)
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), score, True)
    assert (got == 0).all()


@pytest.mark.gpu
def test_renormalised_over_tiny_scores():
    """Scores near the smallest normal number, where a score has lost up to two bits (2^-22 of it): no overflow."""
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(5)
    l = -87.0 - 0.7 * torch.rand(20, 16, generator=g)
    idx = torch.rand(20, 16, generator=g).topk(4, dim=1).indices.to(torch.int32)
    dw = torch.randn(20, 4, generator=g) * 1e3
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), dw.to(DEV), "sigmoid", True, 2.5)
    ref, size = gradient(l, idx, dw, "sigmoid", True, 2.5)
    assert (np.abs(got.double().cpu().numpy() - ref) <= (64 + 6 * 4 + 16) * 2.0 ** -24 * size).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("z", GAPS)
def test_softmax(T, E, k, z):
    check(*confident(T, E, k, z, 6), "softmax", False)


@pytest.mark.gpu
def test_softmax_over_every_expert():
    """All chosen: no share is left over, and equal dw have no gradient."""
    from serve_invariant_moe_gb300 import binding
    l = torch.randn(7, 30, generator=torch.Generator().manual_seed(7))
    idx = torch.arange(30, dtype=torch.int32).expand(7, 30).contiguous()
    got = binding.moe_route_select_backward(l.to(DEV), idx.to(DEV), torch.ones(7, 30, device=DEV), "softmax", False)
    assert (got == 0).all()
