"""Stores of the 8-bit block's kernels: every element that a call owns is written, and nothing beside it.

Outputs are views into the middle of larger buffers filled with a NaN pattern that no kernel writes for finite inputs.  After
a call the view holds none of it and the rest nothing else.  Sizes are the ragged ones: partial tiles, odd row lengths, clipped
bulk stores, groups that end inside a slab, rows that end inside a block of 128.
"""
import pytest
import torch

from test_gpu_fp8_block import COUNTS, deq_rows, deq_weight, dot_bound, fp8_values, plan_of, rows_operand, weight_operand, workspace
from test_gpu_fp8_layer import make_block, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 48                       # rows (or elements of a vector) on either side; keeps 16-byte alignment
POISON = {1: (torch.uint8, 0xFF), 2: (torch.int16, 0x7FC1), 4: (torch.int32, 0x7FC00123)}


@pytest.fixture(scope="module", autouse=True)
def _build():
    from serve_invariant_moe_gb300 import build
    build.build()


def bits(t):
    return t.view(POISON[t.element_size()][0])


class Guarded:
    """The view `.t` of an output between poisoned guards."""

    def __init__(self, shape, dtype):
        raw, value = POISON[dtype.itemsize]
        n = shape[0]
        self.buf = torch.full((n + 2 * GUARD, *shape[1:]), value, dtype=raw, device=DEV).view(dtype)
        self.t = self.buf[GUARD:GUARD + n]

    def check(self, name):
        value = POISON[self.buf.element_size()][1]
        b, n = bits(self.buf), self.t.shape[0]
        assert not (b[GUARD:GUARD + n] == value).any(), f"{name}: an element was not written"
        assert (b[:GUARD] == value).all() and (b[GUARD + n:] == value).all(), f"{name}: a store beside the output"


def check_all(outputs):
    torch.cuda.synchronize()
    for name, g in outputs.items():
        g.check(name)


GEMMS = [(1, 1, 16), (3, 100, 144), (17, 384, 400), (33, 130, 2048), (65, 129, 272), (129, 640, 1040), (300, 1001, 656),
         (700, 1004, 272), (700, 1000, 1040), (1301, 1003, 144), (641, 2048, 512), (2000, 8, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K, dtype):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(M + N)
    (a, sa), (b, sb) = rows_operand(M, K, g), weight_operand(N, K, g)
    out = Guarded((M, N), dtype)
    binding.fp8_gemm(a.to(DEV), sa.to(DEV), b.to(DEV), sb.to(DEV), workspace(), out_dtype=dtype, out=out.t)
    check_all(dict(out=out))


# the last three take the row kernel in gate/up, the first two of them in a wide enough down projection as well
GROUPS = COUNTS + [[100] * 8, [97, 0, 160, 128, 33, 300], [257, 31, 96]]


@pytest.mark.parametrize("H,F", [(144, 256), (1040, 384)])
@pytest.mark.parametrize("counts", GROUPS)
def test_grouped_swiglu(counts, H, F):
    from serve_invariant_moe_gb300 import binding
    E, S = len(counts), sum(counts)
    g = torch.Generator().manual_seed(S + H)
    a, sa = rows_operand(S, H, g)
    w13, s13 = fp8_values((E, 2 * F, H), g), torch.rand(E, 2 * F // 128, (H + 127) // 128, generator=g) * 0.01 + 0.001
    h, hs = Guarded((S, F), torch.float8_e4m3fn), Guarded((S, F // 128), torch.float32)
    binding.moe_grouped_swiglu_fp8(a.to(DEV), sa.to(DEV), plan_of(counts).to(DEV), w13.to(DEV), s13.to(DEV), S, 1,
                                   workspace(), h=h.t, h_scale=hs.t)
    check_all(dict(h=h, h_scale=hs))


# H = 1744 and 2048 give the row kernel enough tiles; a row of 1744 ends inside a tile and inside a bulk store's 32 columns
@pytest.mark.parametrize("H,F", [(144, 256), (1040, 384), (1744, 256), (2048, 128)])
@pytest.mark.parametrize("counts", GROUPS)
def test_grouped_down_in_and_beside_its_rows(counts, H, F):
    """Also against 64 bits: the row kernel's grouped product through bulk stores, with groups of whole and partial slabs."""
    from serve_invariant_moe_gb300 import binding
    E, S = len(counts), sum(counts)
    g = torch.Generator().manual_seed(S * 3 + H)
    a, sa = rows_operand(S, F, g)
    ws = [weight_operand(H, F, g) for _ in range(E)]
    w2, s2 = torch.stack([w for w, _ in ws]), torch.stack([s for _, s in ws])
    y = Guarded((S, H), torch.float32)
    binding.moe_grouped_down_fp8(a.to(DEV), sa.to(DEV), plan_of(counts).to(DEV), w2.to(DEV), s2.to(DEV), S, 1, workspace(),
                                 y=y.t)
    check_all(dict(y=y))
    A, got, first = deq_rows(a, sa), y.t.double().cpu().numpy(), 0
    for e, n in enumerate(counts):
        rows = slice(first, first + n)
        first += n
        W = deq_weight(w2[e], s2[e])
        assert (abs(got[rows] - A[rows] @ W.T) <= dot_bound(A[rows], W, F)).all()


@pytest.mark.parametrize("T,H,E,k", [(1, 16, 4, 1), (5, 144, 8, 3), (200, 2064, 16, 8), (33, 6144, 64, 32)])
def test_routing_and_permutes(T, H, E, k):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T + H)
    q, s = (t.to(DEV) for t in rows_operand(T, H, g))
    logits = torch.randn(T, E, generator=g).to(DEV)
    ws = binding.new_workspace(binding.workspace_size(T, 64, E, k))
    idx, w, plan = Guarded((T, k), torch.int32), Guarded((T, k), torch.float32), Guarded((2 * E + 1 + 2 * T * k,), torch.int32)
    binding.moe_route_select(logits, k, topk_idx=idx.t, topk_w=w.t, plan=plan.t, workspace=ws)
    xp, xs = Guarded((T * k, H), torch.float8_e4m3fn), Guarded((T * k, (H + 127) // 128), torch.float32)
    binding.moe_permute_fp8(q, s, plan.t, E, k, xp.t, xs.t)
    rows = Guarded((T * k, H), torch.bfloat16)
    binding.moe_permute_rows(torch.ones(T, H, dtype=torch.bfloat16, device=DEV), plan.t, E, k, rows.t)
    outputs = dict(idx=idx, w=w, plan=plan, xp=xp, xp_scale=xs, rows=rows)
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            d, d16 = Guarded((T, E), torch.float32), Guarded((T, E), torch.bfloat16)
            binding.moe_route_select_backward(logits, idx.t, w.t, score, renorm, dlogits=d.t, dlogits_bf16=d16.t)
            outputs |= {f"dlogits {score} {renorm}": d, f"dlogits_bf16 {score} {renorm}": d16}
    check_all(outputs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 16), (3, 128), (130, 144), (257, 1040), (2, 140, 160)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(shape, block_rows, dtype):
    from serve_invariant_moe_gb300 import binding
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    rows, cols = shape[-2:]
    blocks = (rows if block_rows == 1 else (rows + 127) // 128, (cols + 127) // 128)
    q, s = Guarded(shape, torch.float8_e4m3fn), Guarded((*shape[:-2], *blocks), torch.float32)
    binding.fp8_quantize(x, block_rows, q=q.t, scale=s.t)
    check_all(dict(q=q, scale=s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 144), (700, 400), (5, 2064), (460, 6160), (7, 16400)])
def test_norm_and_backward(T, H, dtype):
    from serve_invariant_moe_gb300 import binding
    g = torch.Generator().manual_seed(T)
    x, res = (torch.randn(T, H, generator=g).to(dtype).to(DEV) for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    o = dict(residual_out=Guarded((T, H), dtype), out=Guarded((T, H), torch.bfloat16), q=Guarded((T, H), torch.float8_e4m3fn),
             scale=Guarded((T, (H + 127) // 128), torch.float32), rstd=Guarded((T,), torch.float32))
    binding.add_rms_norm(x, w, res, fp8=True, **{name: b.t for name, b in o.items()})
    check_all(o)
    n = binding.rms_norm_backward_workspace_size(T, H)
    space = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    b = dict(dx=Guarded((T, H), dtype), dweight=Guarded((H,), torch.float32))
    binding.add_rms_norm_backward(x, o["residual_out"].t, w, o["rstd"].t, workspace=space[:n],
                                  **{name: v.t for name, v in b.items()})
    check_all(b)
    assert (space[n:] == 0xFF).all()


@pytest.mark.parametrize("B", [0, 1, 3])
def test_decode_of_fewer_requests_than_the_buffers_hold(B):
    blk = make_block(E=32, H=320, F=256, k=6, n_group=8, topk_group=3)
    w, most = blk.w, 9
    x, res = tokens(most, w.H)
    blk.decode(x, res)
    rows = dict(norm=B, q=B, q_scale=B, rstd=B, logits=B, topk_idx=B, topk_w=B, xp=B * w.k, xp_scale=B * w.k, h=B * w.k,
                h_scale=B * w.k, y=B * w.k, hs=B, hs_scale=B, ys=B, residual=B, out=B, plan=2 * w.E + 1 + 2 * B * w.k)
    bufs = {name: t for name, t in blk._bufs.items() if isinstance(t, torch.Tensor) and name != "ws"}
    assert set(bufs) == set(rows)
    for t in bufs.values():
        bits(t).fill_(POISON[t.element_size()][1])
    blk.decode(x[:B], res[:B])
    blk.check()
    for name, t in bufs.items():
        value = POISON[t.element_size()][1]
        assert not (bits(t)[:rows[name]] == value).any(), f"{name}: an element was not written"
        assert (bits(t)[rows[name]:] == value).all(), f"{name}: a store beside the output"
