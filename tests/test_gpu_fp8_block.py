"""The 8-bit block's products, quantisation and permute on the GPU against plain 64-bit computations.

Tolerances.  A product is sum_kb s_kb * p_kb with p_kb an fp32-accumulated dot product of exact e4m3 products and one
fp32 fused multiply-add per block: |error| <= 2 K 2^-24 sum |a||b| (the framework's bound for an fp32-accumulated dot
product, with its slack of 2; the scale product's rounding, 2^-24 relative, is inside it).  A bf16 output adds its own
rounding, 2^-8 of its value at most.  h is held in e4m3: a value within that fp32 bound of a rounding boundary may take
either neighbour, so h is compared after dequantisation, to one e4m3 step of its value (2^-3) plus the step at zero.
"""
import numpy as np
import pytest
import torch

from helpers import dot_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def fp8_values(shape, gen, std=100.0):
    return (torch.randn(shape, generator=gen) * std).clamp(-448, 448).to(torch.float8_e4m3fn)


def rows_operand(M, K, gen):
    return fp8_values((M, K), gen), torch.rand(M, (K + 127) // 128, generator=gen) * 0.02 + 0.001


def weight_operand(N, K, gen):
    return fp8_values((N, K), gen), torch.rand((N + 127) // 128, (K + 127) // 128, generator=gen) * 0.01 + 0.001


def deq_rows(q, s):
    cols = q.shape[-1]
    return (q.double() * s.double().repeat_interleave(128, -1)[..., :cols]).numpy()


def deq_weight(q, s):
    rows, cols = q.shape
    full = s.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return (q.double() * full).numpy()


def workspace():
    from serve_invariant_moe_gb300 import binding
    return binding.new_workspace(256)


GEMM_SIZES = [(1, 128, 128), (1, 1, 16), (3, 100, 144), (16, 256, 256), (17, 384, 400), (33, 130, 2048), (64, 512, 16),
              (65, 129, 272), (129, 640, 1040), (300, 1001, 656), (513, 66, 4096), (1000, 2047, 512)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", GEMM_SIZES)
def test_gemm_matches_64_bits(M, N, K, out_dtype):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(M * 7 + N * 3 + K)
    a, sa = rows_operand(M, K, g)
    b, sb = weight_operand(N, K, g)
    ws = workspace()
    out = binding.fp8_gemm(a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV), ws, out_dtype=out_dtype)
    binding.check_status(ws)
    A, B = deq_rows(a, sa), deq_weight(b, sb)
    ref = A @ B.T
    tol = dot_bound(A, B, K)
    if out_dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert out.shape == (M, N) and (err <= tol).all(), f"max err / bound {np.max(err / tol):.3f}"


def test_gemm_without_rows():
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(1)
    b, sb = weight_operand(64, 128, g)
    a = torch.empty(0, 128, dtype=torch.float8_e4m3fn, device=DEV)
    out = binding.fp8_gemm(a, torch.empty(0, 1, device=DEV), b.to(DEV), sb.to(DEV), workspace())
    assert out.shape == (0, 64)


@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 64, 100, 128, 200, 700])
def test_a_rows_bits_do_not_depend_on_the_batch(M):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(5)
    a, sa = rows_operand(1000, 1168, g)
    b, sb = weight_operand(400, 1168, g)
    a, sa, b, sb = a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV)
    ws = workspace()
    whole = binding.fp8_gemm(a, sa, b, sb, ws, out_dtype=torch.float32)
    first = 1000 - M
    part = binding.fp8_gemm(a[first:].contiguous(), sa[first:].contiguous(), b, sb, ws, out_dtype=torch.float32)
    binding.check_status(ws)
    assert torch.equal(part, whole[first:])


# enough tiles for the row kernel; row lengths that its bulk stores clip, or that keep it from them, in either type
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(700, 1004, 272), (700, 1000, 1040), (1301, 1003, 144), (640, 2048, 512)])
def test_gemm_of_many_rows(M, N, K, out_dtype):
    test_gemm_matches_64_bits(M, N, K, out_dtype)


@pytest.mark.parametrize("M", [1, 16, 50, 128, 129, 333])
def test_a_rows_bits_do_not_depend_on_the_kernel(M):
    """1200 columns: 1000 rows take the row tiles, few rows the column tiles."""
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(8)
    a, sa = rows_operand(1000, 1168, g)
    b, sb = weight_operand(1200, 1168, g)
    a, sa, b, sb = a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV)
    for out_dtype in (torch.float32, torch.bfloat16):
        whole = binding.fp8_gemm(a, sa, b, sb, workspace(), out_dtype=out_dtype)
        part = binding.fp8_gemm(a[500:500 + M].contiguous(), sa[500:500 + M].contiguous(), b, sb, workspace(),
                                out_dtype=out_dtype)
        assert torch.equal(part, whole[500:500 + M])


def test_outputs_of_several_streams():
    """Calls on two streams at once, on inputs made on each: nothing is shared but read-only weights."""
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(12)
    b, sb = (t.to(DEV) for t in weight_operand(600, 512, g))
    inputs = [rows_operand(M, 512, g) for M in (40, 900)]
    want = [binding.fp8_gemm(a.to(DEV), s.to(DEV), b, sb, workspace()) for a, s in inputs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in inputs], []
    spaces = [workspace() for _ in inputs]
    torch.cuda.synchronize()
    for (a, s), stream, ws in zip(inputs, streams, spaces):
        with torch.cuda.stream(stream):
            ad, sd = a.to(DEV), s.to(DEV)
            got.append([binding.fp8_gemm(ad, sd, b, sb, ws) for _ in range(5)])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def test_nan_and_zero_scales_stay_in_their_row():
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(6)
    a, sa = rows_operand(40, 512, g)
    b, sb = weight_operand(200, 512, g)
    ref = binding.fp8_gemm(a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV), workspace(), out_dtype=torch.float32)
    a.view(torch.uint8)[7, 300] = 0x7F          # e4m3 NaN
    sa[9] = 0.0
    sa[11, 2] = float("inf")
    out = binding.fp8_gemm(a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV), workspace(), out_dtype=torch.float32)
    assert torch.isnan(out[7]).all() and (out[9] == 0).all() and not torch.isfinite(out[11]).any()
    keep = [i for i in range(40) if i not in (7, 9, 11)]
    assert torch.equal(out[keep], ref[keep])


# counts per expert: none, one, below / at / above the 16-token step, above one chunk of 128, all in one expert
COUNTS = [[0, 1, 16, 17, 0, 40], [5], [0, 0, 300, 0], [129, 0, 128, 1], [1] * 40, [2, 0, 0, 65, 31, 200, 0]]


def plan_of(counts):
    S = sum(counts)
    c = torch.tensor(counts, dtype=torch.int64)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), c.cumsum(0)])
    rows = torch.arange(S)
    return torch.cat([c, off, rows, rows]).to(torch.int32)


def swiglu_ref(A, W, F):
    g, u = A @ W[:F].T, A @ W[F:].T
    return g / (1.0 + np.exp(-g)) * u


@pytest.mark.parametrize("H,F", [(256, 128), (144, 256), (1040, 384)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_swiglu(counts, H, F):
    from serve_invariant_moe_gb300 import binding
    E, S = len(counts), sum(counts)
    g = torch.Generator().manual_seed(S + H + F)
    a, sa = rows_operand(S, H, g)
    ws = [weight_operand(2 * F, H, g) for _ in range(E)]
    w13 = torch.stack([w for w, _ in ws])
    s13 = torch.stack([s for _, s in ws])
    w = workspace()
    r = binding.moe_grouped_swiglu_fp8(a.to(DEV), sa.to(DEV), plan_of(counts).to(DEV), w13.to(DEV), s13.to(DEV), S, 1, w)
    binding.check_status(w)
    h, hs = r["h"].cpu(), r["h_scale"].cpu()
    A = deq_rows(a, sa)
    first = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        rows = slice(first, first + n)
        first += n
        W = deq_weight(w13[e], s13[e])
        ref = swiglu_ref(A[rows], W, F)
        amax = np.abs(ref).reshape(n, F // 128, 128).max(-1)
        got_s = hs[rows].double().numpy()
        # h = silu(g) u: errors of g and u times the other factor's size (|silu'| <= 1.1, |silu(g)| <= |g|), then 4 roundings
        G, U = np.abs(A[rows] @ W[:F].T), np.abs(A[rows] @ W[F:].T)
        bg, bu = dot_bound(A[rows], W[:F], H), dot_bound(A[rows], W[F:], H)
        bound = 1.1 * bg * (U + bu) + (G + bg) * bu + 2.0 ** -21 * np.abs(ref)
        bmax = bound.reshape(n, F // 128, 128).max(-1)
        assert (np.abs(got_s * 448 - amax) <= bmax + 2.0 ** -22 * amax).all()
        got = deq_rows(h[rows], hs[rows])
        step = np.abs(ref) * 2.0 ** -3 + np.repeat(got_s, 128, 1) * 2.0 ** -9
        assert (np.abs(got - ref) <= step + bound).all()
        # and where no boundary is near, the exact value
        exact = torch.from_numpy(ref / np.repeat(got_s, 128, 1)).float().clamp(-448, 448).to(torch.float8_e4m3fn)
        assert (exact.view(torch.uint8) != h[rows].view(torch.uint8)).float().mean() < 1e-2


@pytest.mark.parametrize("H,F", [(256, 128), (144, 256), (1040, 384)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_down(counts, H, F):
    from serve_invariant_moe_gb300 import binding
    E, S = len(counts), sum(counts)
    g = torch.Generator().manual_seed(S * 3 + H + F)
    a, sa = rows_operand(S, F, g)
    ws = [weight_operand(H, F, g) for _ in range(E)]
    w2 = torch.stack([w for w, _ in ws])
    s2 = torch.stack([s for _, s in ws])
    w = workspace()
    y = binding.moe_grouped_down_fp8(a.to(DEV), sa.to(DEV), plan_of(counts).to(DEV), w2.to(DEV), s2.to(DEV), S, 1, w)
    binding.check_status(w)
    y = y.double().cpu().numpy()
    A = deq_rows(a, sa)
    first = 0
    for e, n in enumerate(counts):
        rows = slice(first, first + n)
        first += n
        W = deq_weight(w2[e], s2[e])
        assert (np.abs(y[rows] - A[rows] @ W.T) <= dot_bound(A[rows], W, F)).all()


def test_grouped_down_of_many_experts():
    """460 experts of 70 rows: the prefix sums of so many groups leave no room for the bulk stores' staging."""
    from serve_invariant_moe_gb300 import binding
    E, n, H, F = 460, 70, 64, 128
    g = torch.Generator().manual_seed(3)
    a, sa = rows_operand(E * n, F, g)
    w2 = fp8_values((E, H, F), g)
    s2 = torch.rand(E, 1, 1, generator=g) * 0.01 + 0.001
    ws = workspace()
    y = binding.moe_grouped_down_fp8(a.to(DEV), sa.to(DEV), plan_of([n] * E).to(DEV), w2.to(DEV), s2.to(DEV), E * n, 1, ws)
    binding.check_status(ws)
    A = torch.from_numpy(deq_rows(a, sa)).view(E, n, F)
    W = w2.double() * s2.double()
    bound = 2.0 * F * 2.0 ** -24 * torch.bmm(A.abs(), W.abs().transpose(1, 2)) + 1e-30
    assert ((y.double().cpu().view(E, n, H) - torch.bmm(A, W.transpose(1, 2))).abs() <= bound).all()


@pytest.mark.parametrize("T", [1, 30, 200])
def test_one_expert_without_a_plan(T):
    """A shared expert: the same bits as an expert that a plan gives every row, and as the dense product."""
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T)
    a, sa = (t.to(DEV) for t in rows_operand(T, 272, g))
    w13, s13 = (t.to(DEV).unsqueeze(0) for t in weight_operand(256, 272, g))
    w2, s2 = (t.to(DEV).unsqueeze(0) for t in weight_operand(272, 128, g))
    ws, plan = workspace(), plan_of([T]).to(DEV)
    r = binding.moe_grouped_swiglu_fp8(a, sa, None, w13, s13, T, 1, ws)
    p = binding.moe_grouped_swiglu_fp8(a, sa, plan, w13, s13, T, 1, ws)
    assert torch.equal(r["h"].view(torch.uint8), p["h"].view(torch.uint8)) and torch.equal(r["h_scale"], p["h_scale"])
    y = binding.moe_grouped_down_fp8(r["h"], r["h_scale"], None, w2, s2, T, 1, ws)
    assert torch.equal(y, binding.moe_grouped_down_fp8(r["h"], r["h_scale"], plan, w2, s2, T, 1, ws))
    assert torch.equal(y, binding.fp8_gemm(r["h"], r["h_scale"], w2[0], s2[0], ws, out_dtype=torch.float32))
    binding.check_status(ws)


def test_a_grouped_rows_bits_do_not_depend_on_its_expert_load():
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(9)
    H, F, E = 272, 256, 3
    a, sa = rows_operand(400, H, g)
    ws = [weight_operand(2 * F, H, g) for _ in range(E)]
    w13, s13 = torch.stack([w for w, _ in ws]).to(DEV), torch.stack([s for _, s in ws]).to(DEV)
    want = None
    for n in (1, 16, 30, 130, 390):
        counts = [4, n, 3]
        S = sum(counts)
        rows = torch.cat([torch.arange(10, 14), torch.tensor([0]), torch.arange(5, 4 + n), torch.arange(3)])[:S]
        picked = a.view(torch.uint8)[rows].view(torch.float8_e4m3fn).to(DEV)
        r = binding.moe_grouped_swiglu_fp8(picked, sa[rows].to(DEV), plan_of(counts).to(DEV), w13, s13, S, 1,
                                           workspace())
        got = (r["h"][4].view(torch.uint8).cpu(), r["h_scale"][4].cpu())
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def quantised(x, block_rows):
    """The definition, in fp32: every step is one correctly rounded operation."""
    x = x.float()
    rows, cols = x.shape
    p = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % block_rows))
    b = p.view(p.shape[0] // block_rows, block_rows, p.shape[1] // 128, 128)
    scale = (b.abs().amax((1, 3)) / 448.0).clamp_min(2.0 ** -126)
    q = (b * (1.0 / scale)[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(p.shape)[:rows, :cols], scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (130, 144), (257, 1040), (1, 8192), (300, 400)])
def test_quantize_is_the_definition(rows, cols, block_rows, dtype):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)
    x[0] = 0.0                                  # a row of zeros
    if rows > 2:
        x[1, :] = 1e-42                         # below the smallest scale
    x = x.to(dtype)
    q, s = binding.fp8_quantize(x.to(DEV), block_rows)
    rq, rs = quantised(x, block_rows)
    assert torch.equal(s.cpu(), rs) and torch.equal(q.float().cpu(), rq.float())


def test_quantize_banks_and_special_values():
    from serve_invariant_moe_gb300 import binding
    x = torch.randn(3, 140, 160, generator=torch.Generator().manual_seed(2))
    q, s = binding.fp8_quantize(x.to(DEV), 128)
    assert s.shape == (3, 2, 2)
    for b in range(3):
        rq, rs = quantised(x[b], 128)
        assert torch.equal(s[b].cpu(), rs) and torch.equal(q[b].float().cpu(), rq.float())
    y = torch.ones(2, 256)
    y[0, 3], y[1, 200] = float("nan"), float("inf")
    q, s = binding.fp8_quantize(y.to(DEV))
    q, s = q.float().cpu(), s.cpu()
    assert torch.isnan(q[0, 3]) and (q[0, :3] == 448).all() and s[0, 0] == np.float32(1.0) / np.float32(448.0)
    assert torch.isinf(s[1, 1]) and torch.isnan(q[1, 200]) and (q[1, 128:200] == 0).all() and (q[1, :128] == 448).all()


@pytest.mark.parametrize("T,H,E,k", [(1, 16, 4, 1), (5, 144, 8, 3), (200, 2064, 16, 8), (33, 6144, 64, 32)])
def test_permute_is_a_copy(T, H, E, k):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T + H)
    q, s = (t.to(DEV) for t in rows_operand(T, H, g))
    logits = torch.randn(T, E, generator=g).to(DEV)
    ws = binding.new_workspace(binding.workspace_size(T, 64, E, k))
    r = binding.moe_route_select(logits, k, plan=True, workspace=ws)
    xp, xs = binding.moe_permute_fp8(q, s, r["plan"], E, k)
    plan = r["plan"].cpu().long()
    off, row_token = plan[E:2 * E + 1], plan[2 * E + 1:2 * E + 1 + T * k]
    assert torch.equal(xp.view(torch.uint8).cpu(), q.view(torch.uint8).cpu()[row_token])
    assert torch.equal(xs.cpu(), s.cpu()[row_token])
    # the plan: experts in order, tokens ascending inside one, every (token, expert) once
    idx = r["topk_idx"].cpu().long()
    assert off[-1] == T * k
    for e in range(E):
        want = (idx == e).any(1).nonzero().reshape(-1)
        assert torch.equal(row_token[off[e]:off[e + 1]], want)


def test_refusals():
    from serve_invariant_moe_gb300 import binding
    from serve_invariant_moe_gb300._lib import InvmoeError
    g = torch.Generator().manual_seed(1)
    a, sa = (t.to(DEV) for t in rows_operand(8, 256, g))
    b, sb = (t.to(DEV) for t in weight_operand(128, 256, g))
    ws = workspace()
    for bad in [dict(a=a.to(torch.bfloat16)), dict(a=a.cpu()), dict(a=a.t()), dict(a_scale=sa[:, :1].contiguous()),
                dict(b=b[:, :128].contiguous()), dict(b_scale=sb[:, :1].contiguous()), dict(out_dtype=torch.float16),
                dict(out=torch.empty(8, 127, dtype=torch.bfloat16, device=DEV)), dict(workspace=ws.cpu())]:
        args = dict(a=a, a_scale=sa, b=b, b_scale=sb, workspace=ws) | bad
        with pytest.raises(ValueError):
            binding.fp8_gemm(**args)
    with pytest.raises(InvmoeError) as e:
        binding.fp8_gemm(a[:, :136].contiguous(), sa, b[:, :136].contiguous(), sb, ws)
    assert e.value.code == -2
    with pytest.raises(InvmoeError) as e:
        binding.fp8_gemm(a, sa, b, sb, ws[:16])
    assert e.value.code == -3
    with pytest.raises(InvmoeError) as e:
        binding.fp8_gemm(torch.zeros(8 * 256 + 1, dtype=torch.uint8, device=DEV)[1:].view(torch.float8_e4m3fn).view(8, 256),
                         sa, b, sb, ws)
    assert e.value.code == -4
    w13, s13 = b.unsqueeze(0), sb.unsqueeze(0)                      # F = 64: not a multiple of 128
    with pytest.raises((InvmoeError, ValueError)):
        binding.moe_grouped_swiglu_fp8(a, sa, None, w13, s13, 8, 1, ws)
    with pytest.raises(ValueError, match="plan"):
        binding.moe_grouped_down_fp8(a[:, :128].contiguous(), sa[:, :1].contiguous(), None,
                                     torch.zeros(2, 128, 128, device=DEV).to(torch.float8_e4m3fn),
                                     torch.ones(2, 1, 1, device=DEV), 8, 1, ws)
    with pytest.raises(ValueError):
        binding.fp8_quantize(torch.zeros(4, 128, dtype=torch.float16, device=DEV))
    with pytest.raises(InvmoeError) as e:
        binding.fp8_quantize(torch.zeros(4, 128, device=DEV), 64, scale=torch.empty(1, 1, device=DEV))
    assert e.value.code == -1
