"""Residual addition + RMSNorm (bf16 and e4m3 outputs) and its backward on the GPU against 64-bit formulas.

Tolerances.  The row r is exact up to its stored type (compared bit by bit with one fp32 addition and one rounding).
rstd: a mean of H squares in fp32, each sum of at most 8V + 5 + 32 terms in a row (V <= 4), so within 80 * 2^-24
relative; y adds 3 roundings: 1e-5 relative covers both.  A bf16 output adds 2^-8 of its value, an e4m3 one a step
(2^-3 of its value, or the step at zero).  Backward: mean(g n) has the same sum error relative to mean |g n|; dweight sums
T terms: T 2^-24 sum |dy n| bounds any order.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
WIDTHS = [16, 48, 128, 144, 1040, 2048, 2064, 6144, 16384, 16400, 32768]


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def inputs(T, H, x_dtype, res_dtype, seed=0):
    g = torch.Generator().manual_seed(seed + T + H)
    x = torch.randn(T, H, generator=g).to(x_dtype)
    res = None if res_dtype is None else (2 * torch.randn(T, H, generator=g)).to(res_dtype)
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16)
    return x, res, w


def check_norm(got, x, res, w):
    r = x.float() if res is None else (x.float() + res.float()).to(res.dtype)
    if res is not None:
        assert torch.equal(got["residual"].cpu(), r)
    r = r.double().numpy()
    rstd = 1 / np.sqrt((r * r).mean(1) + EPS)
    assert np.allclose(got["rstd"].double().cpu().numpy(), rstd, rtol=1e-5, atol=0)
    y = r * rstd[:, None] * w.double().numpy()
    if got["out"] is not None:
        err = np.abs(got["out"].double().cpu().numpy() - y)
        assert (err <= np.abs(y) * (2.0 ** -8 + 1e-5) + 1e-38).all()
    if got["q"] is not None:
        T, H = y.shape
        nb = (H + 127) // 128
        amax = np.abs(np.pad(y, ((0, 0), (0, nb * 128 - H)))).reshape(T, nb, 128).max(-1)
        s = got["scale"].double().cpu().numpy()
        assert s.shape == (T, nb) and np.allclose(s, np.maximum(amax / 448, 2.0 ** -126), rtol=2e-5, atol=0)
        full = np.repeat(s, 128, 1)[:, :H]
        d = got["q"].double().cpu().numpy() * full
        assert (np.abs(d - y) <= np.abs(y) * (2.0 ** -4 + 1e-4) + full * 2.0 ** -10 + 1e-38).all()


@pytest.mark.parametrize("x_dtype,res_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                               (torch.float32, torch.bfloat16), (torch.float32, torch.float32),
                                               (torch.bfloat16, None), (torch.float32, None)])
@pytest.mark.parametrize("H", WIDTHS)
def test_norm(H, x_dtype, res_dtype):
    from serve_invariant_moe_gb300 import binding
    x, res, w = inputs(3, H, x_dtype, res_dtype)
    got = binding.add_rms_norm(x.to(DEV), w.to(DEV), None if res is None else res.to(DEV), eps=EPS, fp8=True)
    check_norm(got, x, res, w)


@pytest.mark.parametrize("T", [0, 1, 2, 700])
@pytest.mark.parametrize("out,fp8", [(True, False), (False, True), (True, True)])
def test_norm_batches_and_outputs(T, out, fp8):
    from serve_invariant_moe_gb300 import binding
    x, res, w = inputs(T, 400, torch.bfloat16, torch.bfloat16)
    res_dev = res.to(DEV)
    got = binding.add_rms_norm(x.to(DEV), w.to(DEV), res_dev, eps=EPS, out=out, fp8=fp8, residual_out=res_dev)  # in place
    assert got["residual"].data_ptr() == res_dev.data_ptr()
    assert (got["out"] is not None) == out and (got["q"] is not None) == fp8
    if T:
        check_norm(got, x, res, w)


def test_a_rows_bits_do_not_depend_on_the_batch():
    from serve_invariant_moe_gb300 import binding
    x, res, w = inputs(200, 2064, torch.float32, torch.bfloat16)
    x, res, w = x.to(DEV), res.to(DEV), w.to(DEV)
    a = binding.add_rms_norm(x, w, res, fp8=True)
    b = binding.add_rms_norm(x[150:151].contiguous(), w, res[150:151].contiguous(), fp8=True)
    for name in ("residual", "out", "scale", "rstd"):
        assert torch.equal(a[name][150:151], b[name]), name
    assert torch.equal(a["q"][150:151].view(torch.uint8), b["q"].view(torch.uint8))


def test_norm_special_rows():
    """A row of zeros, and rows with a NaN or an infinity, stay in their own row."""
    from serve_invariant_moe_gb300 import binding
    x, _, w = inputs(5, 256, torch.float32, None)
    x[0] = 0.0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] *= 1e-30
    got = binding.add_rms_norm(x.to(DEV), w.to(DEV), eps=EPS, fp8=True)
    out, q, s = got["out"].cpu(), got["q"].float().cpu(), got["scale"].cpu()
    assert (out[0] == 0).all() and (q[0] == 0).all() and (s[0] == 2.0 ** -126).all()
    assert torch.isnan(out[1]).all() and torch.isnan(q[1]).all()
    assert got["rstd"][2] == 0 and torch.isnan(out[2, 9]) and (out[2, :9] == 0).all()
    assert torch.isfinite(out[3:]).all() and torch.isfinite(q[3:]).all()
    ref = binding.add_rms_norm(x[4:].to(DEV), w.to(DEV), eps=EPS)
    assert torch.equal(ref["out"].cpu(), out[4:])


def grads64(dy, r, w, rstd, dres):
    r, dy, w = r.double().numpy(), dy.double().numpy(), w.double().numpy()
    rs = rstd.double().numpy()[:, None]
    n, g = r * rs, dy * w
    dx = rs * (g - n * (g * n).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres.double().numpy()
    return dx, (dy * n).sum(0), n, g


def test_the_backward_formula_against_differences():
    """The formula itself, in 64 bits: central differences of sum(dy * norm(r)) in every coordinate."""
    g = torch.Generator().manual_seed(3)
    T, H = 2, 16
    r, dy = torch.randn(T, H, generator=g).double(), torch.randn(T, H, generator=g).double()
    w = (1 + 0.2 * torch.randn(H, generator=g)).double()
    rstd = 1 / (r.square().mean(1) + EPS).sqrt()
    dx, dw, _, _ = grads64(dy, r, w, rstd, None)

    def f(r, w):
        return float((dy * r / (r.square().mean(1, keepdim=True) + EPS).sqrt() * w).sum())
    h = 1e-6
    for t in range(T):
        for i in range(H):
            d = torch.zeros_like(r)
            d[t, i] = h
            assert abs((f(r + d, w) - f(r - d, w)) / (2 * h) - dx[t, i]) < 1e-7
    for i in range(H):
        d = torch.zeros_like(w)
        d[i] = h
        assert abs((f(r, w + d) - f(r, w - d)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.parametrize("x_dtype,dy_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                              (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("T,H", [(1, 16), (2, 144), (5, 2048), (700, 400), (3, 6144), (1300, 48), (2, 32768)])
@pytest.mark.parametrize("with_dres", [False, True])
def test_norm_backward(T, H, x_dtype, dy_dtype, with_dres):
    from serve_invariant_moe_gb300 import binding
    x, dres, w = inputs(T, H, x_dtype, x_dtype, seed=4)
    dres = dres if with_dres else None
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(dy_dtype)
    rstd = binding.add_rms_norm(x.to(DEV), w.to(DEV), eps=EPS)["rstd"]
    got = binding.add_rms_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), rstd,
                                        dres=None if dres is None else dres.to(DEV))
    dx, dw, n, g = grads64(dy, x, w, rstd.cpu(), dres)
    rs = rstd.double().cpu().numpy()[:, None]
    scale = rs * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    tol = 1e-5 * scale + (2.0 ** -8 if x_dtype == torch.bfloat16 else 2.0 ** -22) * np.abs(dx)
    assert got["dx"].dtype == x_dtype and (np.abs(got["dx"].double().cpu().numpy() - dx) <= tol + 1e-30).all()
    dtol = (T + 4) * 2.0 ** -24 * np.abs(dy.double().numpy() * n).sum(0) + 1e-30
    assert (np.abs(got["dweight"].double().cpu().numpy() - dw) <= dtol).all()
    # the same bits again, and without dweight, and into dres itself
    again = binding.add_rms_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), rstd,
                                          dres=None if dres is None else dres.to(DEV))
    assert torch.equal(got["dx"], again["dx"]) and torch.equal(got["dweight"], again["dweight"])
    buf = None if dres is None else dres.to(DEV)
    only = binding.add_rms_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), rstd, dres=buf, dx=buf, dweight=False)
    assert only["dweight"] is None and torch.equal(only["dx"], got["dx"])


@pytest.mark.parametrize("x_dtype,dy_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,H", [(400, 10256), (333, 4112), (160, 8192)])
def test_norm_backward_of_wide_rows(T, H, x_dtype, dy_dtype):
    """Several rows a block where a row needs two or four vectors a thread."""
    test_norm_backward(T, H, x_dtype, dy_dtype, True)


def test_backward_without_rows_clears_dweight():
    from serve_invariant_moe_gb300 import binding
    z = torch.empty(0, 64, device=DEV)
    got = binding.add_rms_norm_backward(z, z, torch.ones(64, dtype=torch.bfloat16, device=DEV), torch.empty(0, device=DEV))
    assert (got["dweight"] == 0).all()


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    x, res, w = (t.to(DEV) for t in inputs(4, 128, torch.bfloat16, torch.bfloat16))
    for bad in [dict(x=x.half()), dict(x=x.cpu()), dict(x=x.t()), dict(weight=w.float()), dict(weight=w[:64]),
                dict(residual=res[:2]), dict(residual=res.half()), dict(residual=None, residual_out=res),
                dict(out=torch.empty(4, 128, device=DEV)), dict(fp8=True, scale=torch.empty(4, 2, device=DEV))]:
        with pytest.raises(ValueError):
            binding.add_rms_norm(**(dict(x=x, weight=w, residual=res) | bad))
    for bad, code in [(dict(x=torch.zeros(2, 24, device=DEV), weight=w[:24]), -2), (dict(eps=-1.0), -1),
                      (dict(out=False), -1), (dict(eps=float("nan")), -1)]:
        with pytest.raises(InvmoeError) as e:
            binding.add_rms_norm(**(dict(x=x, weight=w) | bad))
        assert e.value.code == code
    rstd = torch.ones(4, device=DEV)
    with pytest.raises(ValueError):
        binding.add_rms_norm_backward(x, x, w, rstd[:2])
    with pytest.raises(ValueError):
        binding.add_rms_norm_backward(x, x, w, rstd, dres=res.float())
    with pytest.raises(InvmoeError) as e:
        binding.add_rms_norm_backward(x, x, w, rstd, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    assert e.value.code == -3
