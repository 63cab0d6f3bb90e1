"""The norms after and before a block (sandwich_norm) and their backward on the GPU against 64-bit formulas and differences.

Tolerances.  A sum over a row has at most 8V + 5 + 32 terms after one another in fp32 (V <= 4), so a mean of squares is within
80 * 2^-24 of itself and a mean of signed products within that of the mean of their absolute values: 1e-5 covers both, with the
few roundings of the products around them.  The stored row and every output add half a step of their type
(torch.finfo(t).eps / 2) of their value.  The second norm is checked from the row that the kernel stored.  A sum over T rows
adds T * 2^-24 of the sum of its terms' absolute values.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32
C = 1e-5
TYPES = [(BF, BF), (BF, F32), (F32, BF), (F32, F32)]
WIDTHS = [16, 48, 128, 1040, 2048, 2064, 6144, 8192, 8208, 16400, 32768]


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def half(t):
    return torch.finfo(t).eps / 2


def inputs(T, H, xt, rt, gate, seed=0):
    g = torch.Generator().manual_seed(seed + T + H)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    a = dict(x=(0.5 * r(T, H)).to(xt), w_post=(1 + 0.2 * r(H)).to(BF), residual=(2 * r(T, H)).to(rt),
             w_next=(1 + 0.2 * r(H)).to(BF), gate=None)
    if gate == "channel":
        a["gate"] = (0.5 + 0.3 * r(H)).to(BF)
    elif gate == "token":
        a["gate"] = torch.sigmoid(r(T))
    return {n: None if t is None else t.to(DEV) for n, t in a.items()}


def factor(a, b):
    if a["gate"] is None:
        return torch.tensor(b, dtype=torch.float64, device=DEV)
    g = a["gate"].double() * b
    return g[:, None] if a["gate"].dtype == F32 else g[None]


def check_forward(got, a, rs=1.0, bs=1.0, eps=EPS):
    x, res = a["x"].double(), a["residual"].double()
    rstd = (x.square().mean(-1) + eps).rsqrt()
    assert torch.allclose(got["rstd_post"].double(), rstd, rtol=C, atol=0)
    branch = x * rstd[:, None] * a["w_post"].double() * factor(a, bs)
    want = rs * res + branch
    stored = got["residual"]
    assert stored.dtype == a["residual"].dtype
    err = (stored.double() - want).abs()
    assert (err <= C * (branch.abs() + (rs * res).abs()) + half(stored.dtype) * want.abs() + 1e-38).all()
    if a["w_next"] is None:
        assert got["out"] is None and got["rstd"] is None and got["q"] is None
        return
    r = stored.double()
    rstd = (r.square().mean(-1) + eps).rsqrt()
    assert torch.allclose(got["rstd"].double(), rstd, rtol=C, atol=0)
    y = r * rstd[:, None] * a["w_next"].double()
    if got["out"] is not None:
        assert ((got["out"].double() - y).abs() <= y.abs() * (half(BF) + C) + 1e-38).all()
    if got["q"] is not None:
        T, H = y.shape
        nb = (H + 127) // 128
        amax = torch.nn.functional.pad(y, (0, nb * 128 - H)).abs().view(T, nb, 128).amax(-1)
        s = got["scale"].double()
        assert torch.allclose(s, (amax / 448).clamp_min(2.0 ** -126), rtol=2 * C, atol=0)
        s = s.repeat_interleave(128, -1)[:, :H]
        assert ((got["q"].double() * s - y).abs() <= y.abs() * (2.0 ** -4 + 1e-4) + s * 2.0 ** -10).all()


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_forward(H, xt, rt, gate):
    from serve_invariant_moe_gb300 import binding
    a = inputs(3, H, xt, rt, gate)
    check_forward(binding.sandwich_norm(**a, residual_scale=0.875, branch_scale=0.25, fp8=True), a, 0.875, 0.25)


@pytest.mark.parametrize("T", [0, 1, 700])
def test_forward_outputs(T):
    from serve_invariant_moe_gb300 import binding
    a = inputs(T, 400, F32, BF, "token")
    for out, fp8 in ((True, False), (False, True), (True, True)):
        got = binding.sandwich_norm(**a, out=out, fp8=fp8)
        assert (got["out"] is not None) == out and (got["q"] is not None) == fp8
        check_forward(got, a)
    a["w_next"] = None
    got = binding.sandwich_norm(**a)
    check_forward(got, a)
    at = a["residual"].clone()                       # in place
    again = binding.sandwich_norm(**{**a, "residual": at}, residual_out=at)
    assert again["residual"].data_ptr() == at.data_ptr() and torch.equal(again["residual"], got["residual"])


def test_without_gate_and_scales_it_is_the_two_norms():
    """One call against add_rms_norm twice: the same formulas, so no more than the roundings apart; a scale of 0 drops a term."""
    from serve_invariant_moe_gb300 import binding
    a = inputs(9, 2064, F32, F32, None)
    got = binding.sandwich_norm(**a)
    first = binding.add_rms_norm(a["x"], a["w_post"])
    assert torch.equal(first["rstd"], got["rstd_post"])
    second = binding.add_rms_norm(got["residual"], a["w_next"])
    assert torch.equal(second["rstd"], got["rstd"]) and torch.equal(second["out"], got["out"])
    assert torch.equal(binding.sandwich_norm(**a, branch_scale=0.0)["residual"], a["residual"])
    alone = binding.sandwich_norm(**a, residual_scale=0.0)["residual"]
    assert torch.equal(alone.to(BF), first["out"])


def test_a_rows_bits_do_not_depend_on_the_batch():
    from serve_invariant_moe_gb300 import binding
    a = inputs(200, 2064, F32, BF, "token")
    whole = binding.sandwich_norm(**a, fp8=True)
    one = {n: t if t is None or n in ("w_post", "w_next") else t[150:151].contiguous() for n, t in a.items()}
    row = binding.sandwich_norm(**one, fp8=True)
    for name in ("residual", "out", "scale", "rstd", "rstd_post"):
        assert torch.equal(whole[name][150:151], row[name]), name
    assert torch.equal(whole["q"][150:151].view(torch.uint8), row["q"].view(torch.uint8))


def test_special_rows_stay_their_own():
    from serve_invariant_moe_gb300 import binding
    a = inputs(6, 256, F32, F32, "token")
    clean = binding.sandwich_norm(**a)
    a["x"][0] = 0.0
    a["x"][1, 7] = float("nan")
    a["residual"][2, 9] = float("inf")
    a["x"][3] *= 1e-30
    got = binding.sandwich_norm(**a)
    assert torch.equal(got["residual"][0], a["residual"][0])
    assert torch.isnan(got["residual"][1]).all() and torch.isnan(got["out"][1]).all()
    assert torch.isinf(got["residual"][2, 9]) and torch.isfinite(got["residual"][2]).sum() == 255
    for name in ("residual", "out", "rstd", "rstd_post"):
        assert torch.isfinite(got[name][3:].float()).all()
        assert torch.equal(got[name][4:], clean[name][4:])


# ------------------------------------------------------------------------------------------------------- backward

def gradients(T, H, rt, yt, seed=1):
    g = torch.Generator().manual_seed(seed + T + H)
    return (torch.randn(T, H, generator=g).to(yt).to(DEV), torch.randn(T, H, generator=g).to(rt).to(DEV))


def saved(a, rs=1.0, bs=1.0):
    from serve_invariant_moe_gb300 import binding
    f = binding.sandwich_norm(**a, residual_scale=rs, branch_scale=bs)
    return f["rstd_post"], f["residual"], f["rstd"]


def check_backward(got, a, dy, dres, rstd_post, r, rstd, rs=1.0, bs=1.0):
    T, H = a["x"].shape
    w_next = a["w_next"]
    mag = torch.zeros(T, H, dtype=torch.float64, device=DEV)       # of the terms of d
    d = mag.clone()
    if dres is not None:
        d += dres.double()
        mag += dres.double().abs()
    if dy is not None:
        n = r.double() * rstd.double()[:, None]
        e = dy.double() * w_next.double()
        s = rstd.double()[:, None]
        d += s * (e - n * (e * n).mean(-1, keepdim=True))
        mag += s * (e.abs() + n.abs() * (e * n).abs().mean(-1, keepdim=True))
        t = (dy.double() * n)
        assert ((got["dw_next"].double() - t.sum(0)).abs() <= (C + T * 2.0 ** -24) * t.abs().sum(0) + 1e-38).all()
    err = C * mag
    out = got["dresidual"]
    assert out.dtype == a["residual"].dtype
    assert ((out.double() - rs * d).abs() <= abs(rs) * err + half(out.dtype) * (rs * d).abs() + 1e-38).all()
    n = a["x"].double() * rstd_post.double()[:, None]
    w = a["w_post"].double()
    f = factor(a, bs)
    u, du = f * d * w, (f * w).abs() * err
    m, dm = (u * n).mean(-1, keepdim=True), (du * n.abs()).mean(-1, keepdim=True) + C * (u * n).abs().mean(-1, keepdim=True)
    s = rstd_post.double()[:, None]
    dx = s * (u - n * m)
    bound = s * (du + n.abs() * dm) + C * s * (u.abs() + n.abs() * m.abs()) + half(a["x"].dtype) * dx.abs()
    assert got["dx"].dtype == a["x"].dtype
    assert ((got["dx"].double() - dx).abs() <= bound + 1e-38).all()

    def column_sum(name, t, dt):
        assert ((got[name].double() - t.sum(0)).abs() <= dt.sum(0) + (C + T * 2.0 ** -24) * t.abs().sum(0) + 1e-38).all(), name
    column_sum("dw_post", f * d * n, (f * n).abs() * err)
    if a["gate"] is None:
        assert got["dgate"] is None
    elif a["gate"].dtype == BF:
        column_sum("dgate", bs * d * w * n, (bs * w * n).abs() * err)
    else:
        t = bs * d * w * n
        e = (bs * w * n).abs() * err
        assert ((got["dgate"].double() - t.sum(-1)).abs() <= e.sum(-1) + C * t.abs().sum(-1) + 1e-38).all()


@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("T,H", [(5, 16), (37, 144), (1, 1040), (160, 2048), (9, 2064), (311, 400), (6, 8192), (5, 8208),
                                 (3, 32768)])
def test_backward(T, H, yt, xt, rt, gate):
    from serve_invariant_moe_gb300 import binding
    a = inputs(T, H, xt, rt, gate)
    dy, dres = gradients(T, H, rt, yt)
    rstd_post, r, rstd = saved(a, 0.875, 0.25)
    got = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, a["w_next"], rstd, a["gate"], 0.875, 0.25)
    check_backward(got, a, dy, dres, rstd_post, r, rstd, 0.875, 0.25)


@pytest.mark.parametrize("T,H", [(1, 64), (460, 2048), (1000, 6144), (2000, 96), (65, 16400)])
def test_backward_batches(T, H):
    from serve_invariant_moe_gb300 import binding
    a = inputs(T, H, F32, BF, "channel")
    dy, dres = gradients(T, H, BF, BF)
    rstd_post, r, rstd = saved(a)
    args = (a["x"], a["w_post"], rstd_post, r)
    whole = binding.sandwich_norm_backward(dy, dres, *args, a["w_next"], rstd, a["gate"])
    check_backward(whole, a, dy, dres, rstd_post, r, rstd)
    again = binding.sandwich_norm_backward(dy, dres, *args, a["w_next"], rstd, a["gate"])
    rows = binding.sandwich_norm_backward(dy, dres, *args, a["w_next"], rstd, a["gate"], dweights=False)
    assert rows["dw_post"] is None and rows["dw_next"] is None and rows["dgate"] is None
    for name in ("dx", "dresidual"):
        assert torch.equal(whole[name], again[name]) and torch.equal(whole[name], rows[name]), name
    for name in ("dw_post", "dw_next", "dgate"):
        assert torch.equal(whole[name], again[name]), name


@pytest.mark.parametrize("T,H", [(7, 400), (3, 8208)])
def test_backward_of_one_norm_or_without_a_stream_gradient(T, H):
    from serve_invariant_moe_gb300 import binding
    a = inputs(T, H, F32, F32, "token")
    dy, dres = gradients(T, H, F32, BF)
    rstd_post, r, rstd = saved(a)
    got = binding.sandwich_norm_backward(dy, None, a["x"], a["w_post"], rstd_post, r, a["w_next"], rstd, a["gate"])
    check_backward(got, a, dy, None, rstd_post, r, rstd)
    got = binding.sandwich_norm_backward(None, dres, a["x"], a["w_post"], rstd_post, r, gate=a["gate"])
    assert got["dw_next"] is None
    check_backward(got, a, None, dres, rstd_post, r, rstd)


def test_no_rows_have_zero_weight_gradients():
    from serve_invariant_moe_gb300 import binding
    a = inputs(0, 64, F32, F32, "channel")
    dy, dres = gradients(0, 64, F32, F32)
    got = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], torch.empty(0, device=DEV), a["residual"], a["w_next"],
                                         torch.empty(0, device=DEV), a["gate"])
    for name in ("dw_post", "dw_next", "dgate"):
        assert got[name].shape == (64,) and (got[name] == 0).all()


@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_backward_against_differences(gate):
    """Each gradient along a random direction against central differences of the formula in 64 bits."""
    from serve_invariant_moe_gb300 import binding
    T, H, rs, bs = 5, 48, 0.875, 1.25
    a = inputs(T, H, F32, F32, gate)
    dy, dres = gradients(T, H, F32, F32)

    def value(v):
        gate_of = 1.0 if gate is None else v["gate"][None] if gate == "channel" else v["gate"][:, None]
        n = v["x"] * (v["x"].square().mean(-1, keepdim=True) + EPS).rsqrt() * v["w_post"] * gate_of
        r = rs * v["residual"] + bs * n
        y = r * (r.square().mean(-1, keepdim=True) + EPS).rsqrt() * v["w_next"]
        return float((r * dres.double()).sum() + (y * dy.double()).sum())

    rstd_post, r, rstd = saved(a, rs, bs)
    got = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, a["w_next"], rstd, a["gate"], rs, bs)
    at = {n: t.double() for n, t in a.items() if t is not None}
    names = {"x": "dx", "residual": "dresidual", "w_post": "dw_post", "w_next": "dw_next", "gate": "dgate"}
    g = torch.Generator().manual_seed(7)
    for name in at:
        v = torch.randn(at[name].shape, generator=g, dtype=torch.float64).to(DEV)
        h = 1e-4
        want = (value({**at, name: at[name] + h * v}) - value({**at, name: at[name] - h * v})) / (2 * h)
        grad = got[names[name]].double()
        # differences: h^2 times a third derivative, about 1e-8 of it; fp32 gradients: C of their terms
        assert abs(float((grad * v).sum()) - want) <= 10 * C * float(grad.norm() * v.norm()), name


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    a = inputs(4, 64, F32, F32, None)
    with pytest.raises(InvmoeError):
        binding.sandwich_norm(**a, out=False)
    with pytest.raises(ValueError, match="w_next"):
        binding.sandwich_norm(**{**a, "w_next": None}, fp8=True)
    with pytest.raises(ValueError, match="gate"):
        binding.sandwich_norm(**{**a, "gate": torch.ones(5, device=DEV)})
    with pytest.raises(ValueError, match="residual"):
        binding.sandwich_norm(**{**a, "residual": a["residual"][:3]})
    both = torch.zeros(5, 64, device=DEV)
    with pytest.raises(InvmoeError, match="overlaps"):
        binding.sandwich_norm(**{**a, "residual": both[:4]}, residual_out=both[1:])
    with pytest.raises(InvmoeError, match="overlaps"):
        binding.sandwich_norm(**{**a, "x": both[:4]}, residual_out=both[1:])
    dy, dres = gradients(4, 64, F32, F32)
    one = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="together"):
        binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], one, a["residual"])
    with pytest.raises(InvmoeError, match="both NULL"):
        binding.sandwich_norm_backward(None, None, a["x"], a["w_post"], one, a["residual"])
    with pytest.raises(InvmoeError, match="overlaps"):
        binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], one, a["residual"], a["w_next"], one, dx=a["x"])
    with pytest.raises(InvmoeError, match="workspace"):
        binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], one, a["residual"], a["w_next"], one,
                                       workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    assert math.isfinite(float(binding.sandwich_norm(**a)["residual"].sum()))


def test_a_captured_pair_replays_with_other_inputs():
    """Forward and backward in one graph, replayed on new values; eager calls on another stream give the same bits."""
    from serve_invariant_moe_gb300 import binding
    a = inputs(33, 2064, F32, BF, "channel")
    dy, dres = gradients(33, 2064, BF, F32)

    def both():
        f = binding.sandwich_norm(**a)
        b = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], f["rstd_post"], f["residual"], a["w_next"], f["rstd"],
                                           a["gate"])
        return [f["residual"], f["out"], *b.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for seed in (5, 6):
        other = inputs(33, 2064, F32, BF, "channel", seed)
        for n in a:
            a[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            want = both()
        side.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


def test_forward_offsets_past_2_31():
    """The last rows of a matrix of more than 2^31 elements have the bits that they have alone."""
    from serve_invariant_moe_gb300 import binding
    T, H, n = 131_200, 16400, 5
    assert (T - n) * H > 2 ** 31
    small = inputs(n, H, BF, BF, "token")
    whole = {name: torch.zeros(T, *t.shape[1:], dtype=t.dtype, device=DEV) if t.shape[0] == n else t for name, t in small.items()}
    for name, t in small.items():
        if t.shape[0] == n:
            whole[name][-n:] = t
    got, want = (binding.sandwich_norm(**a, residual_scale=0.875, branch_scale=0.25, fp8=True) for a in (whole, small))
    for name, t in want.items():
        t, end = (v.view(torch.uint8) if v.dtype == torch.float8_e4m3fn else v for v in (t, got[name][-n:]))
        assert torch.equal(end, t), name
    assert (got["residual"][:-n] == 0).all()


@pytest.mark.parametrize("T,H", [(262_400, 8192), (131_200, 16400)])
def test_backward_offsets_past_2_31(T, H):
    """Rows without a gradient, but for the last: their gradients are those that they have alone, and so are the weights', up to
    the order of the sum (at most 5 terms and zeros: 5 * 2^-24 of their absolute values, on both sides)."""
    from serve_invariant_moe_gb300 import binding
    n = 5
    assert (T - n) * H > 2 ** 31
    a = inputs(n, H, BF, BF, "token")
    dy, dres = gradients(n, H, BF, BF)
    rstd_post, r, rstd = saved(a)

    def tall(t):
        whole = torch.zeros(T, *t.shape[1:], dtype=t.dtype, device=DEV)
        whole[-n:] = t
        return whole
    names = dict(dweights=True)
    want = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, a["w_next"], rstd, a["gate"], **names)
    got = binding.sandwich_norm_backward(tall(dy), tall(dres), tall(a["x"]), a["w_post"], tall(rstd_post), tall(r), a["w_next"],
                                         tall(rstd), tall(a["gate"]), **names)
    for name in ("dx", "dresidual", "dgate"):
        assert torch.equal(got[name][-n:], want[name]), name
        assert (got[name][:-n] == 0).all(), name
    for name, size in (("dw_post", 64.0), ("dw_next", 64.0)):
        # no term is above `size`: |dy|, |d| below 6 times |n| below 6, times a gate below 1, 5 rows
        assert ((got[name] - want[name]).abs() <= 10 * 2.0 ** -24 * 5 * size).all(), name


def test_backwards_on_two_streams():
    """Each with a workspace that torch allocates on its stream."""
    from serve_invariant_moe_gb300 import binding
    cases = []
    for seed in range(4):
        a = inputs(300, 2064, F32, BF, "channel", seed)
        dy, dres = gradients(300, 2064, BF, F32)
        rstd_post, r, rstd = saved(a)
        args = (dy, dres, a["x"], a["w_post"], rstd_post, r, a["w_next"], rstd, a["gate"])
        cases.append((args, binding.sandwich_norm_backward(*args)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            got.append(binding.sandwich_norm_backward(*cases[i % 4][0]))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for name, t in cases[i % 4][1].items():
            assert torch.equal(g[name], t), (i, name)


@pytest.mark.parametrize("group,two_norms", [(0, True), (1, True), (1, False)])
def test_what_a_wait_that_ran_out_leaves_is_no_gradient(group, two_norms):
    """Blocks of four rows whose second row never comes: the rows before it are right, the others and the weights' gradients are
    NaN, so a caller that reads no status (or gave no workspace to read) does not train on them."""
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    T, H = 1000, 2048                               # 250 blocks
    a = inputs(T, H, F32, F32, None)
    dy, dres = gradients(T, H, F32, F32)
    rstd_post, r, rstd = saved(a)
    w_next = a["w_next"]
    if not two_norms:
        dy = w_next = rstd = None
    ws = binding.new_workspace(binding.sandwich_norm_backward_workspace_size(T, H))
    want = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, w_next, rstd, workspace=ws)
    binding.check_status(ws)
    got = binding.debug_stalled_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, w_next, rstd, group, ws, timeout_us=5000)
    with pytest.raises(InvmoeError) as e:
        binding.check_status(ws)
    assert e.value.code == -6
    for name in ("dx", "dresidual"):
        assert torch.equal(got[name][::4], want[name][::4]), name
        assert all(bool(got[name][i::4].isnan().all()) for i in (1, 2, 3)), name
    assert bool(got["dw_post"].isnan().all())
    assert (got["dw_next"] is None) if not two_norms else bool(got["dw_next"].isnan().all())
    again = binding.sandwich_norm_backward(dy, dres, a["x"], a["w_post"], rstd_post, r, w_next, rstd, workspace=ws)
    binding.check_status(ws)
    for name in ("dx", "dresidual", "dw_post"):
        assert torch.equal(again[name], want[name]), name


@pytest.mark.parametrize("T,H,xt,rt,yt,without", [(4096, 2048, F32, F32, F32, None), (3000, 96, BF, BF, BF, None),
                                                  (1500, 4096, F32, F32, F32, None), (1200, 4608, F32, BF, BF, None),
                                                  (2000, 6144, F32, BF, BF, None), (500, 8192, F32, F32, F32, None),
                                                  (500, 8192, F32, BF, BF, None), (3000, 2048, F32, F32, F32, "dy"),
                                                  (900, 8192, F32, F32, F32, "dres"), (1500, 2064, BF, F32, F32, "dy")])
def test_rows_that_come_through_used_places(T, H, xt, rt, yt, without):
    """More rows to a block than its ring has places, down to a single place (8192 columns, all fp32): a copy that came too early
    would overwrite a row still being read, every one of which has values of its own."""
    from serve_invariant_moe_gb300 import binding
    a = inputs(T, H, xt, rt, "channel")
    dy, dres = gradients(T, H, rt, yt)
    rstd_post, r, rstd = saved(a, 0.875, 0.25)
    w_next = a["w_next"]
    if without == "dy":
        dy = w_next = rstd = None
    elif without == "dres":
        dres = None
    args = (dy, dres, a["x"], a["w_post"], rstd_post, r, w_next, rstd, a["gate"], 0.875, 0.25)
    got = binding.sandwich_norm_backward(*args)
    check_backward(got, a, dy, dres, rstd_post, r, rstd, 0.875, 0.25)
    again = binding.sandwich_norm_backward(*args)
    assert all(torch.equal(got[n], again[n]) for n in got if got[n] is not None)
