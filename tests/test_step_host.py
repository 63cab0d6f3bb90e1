"""CPU-side checks of a drafted decode step's entry points: host-side validation, sizes, refusal of host tensors."""
import collections
import contextlib
import ctypes
import gc
import threading
import types
import weakref

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from serve_invariant_moe_gb300 import build, _lib
    build.build()
    return _lib.lib()


N = None
P = ctypes.c_void_p(4096)          # never read: every call below is refused on the host


def test_sandwich_norm_rejects_before_any_launch(lib):
    f = lib.sandwich_norm
    tail = (1.0, 1.0, 1e-6, P, P, N, N, N, N, N)
    assert f(P, 5, P, P, 0, N, 0, P, 4, 64, *tail) == -1
    assert f(P, 0, P, P, 7, N, 0, P, 4, 64, *tail) == -1
    assert f(P, 0, P, P, 0, N, 0, P, 4, 40, *tail) == -2
    assert f(P, 0, P, P, 0, N, 0, P, 4, 32784, *tail) == -2
    assert f(P, 0, P, P, 0, N, 0, P, -1, 64, *tail) == -1
    assert f(P, 0, P, P, 0, N, 1, P, 4, 64, *tail) == -1 and b"gate" in lib.invmoe_last_error()
    assert f(P, 0, P, P, 0, P, 3, P, 4, 64, *tail) == -1
    assert f(P, 0, P, P, 0, N, 0, N, 4, 64, *tail) == -1 and b"w_next" in lib.invmoe_last_error()
    assert f(P, 0, P, P, 0, N, 0, P, 4, 64, 1.0, 1.0, -1.0, P, P, N, N, N, N, N) == -1
    assert f(P, 0, P, P, 0, N, 0, P, 4, 64, float("nan"), 1.0, 1e-6, P, P, N, N, N, N, N) == -1
    assert f(P, 0, P, P, 0, N, 0, P, 4, 64, 1.0, 1.0, 1e-6, P, P, P, N, N, N, N) == -1 and b"q and scale" in lib.invmoe_last_error()
    assert f(ctypes.c_void_p(4100), 0, P, P, 0, N, 0, P, 4, 64, *tail) == -4
    assert f(P, 0, P, P, 0, N, 0, P, 0, 64, *tail) == 0                     # no rows


def test_sandwich_norm_backward_rejects_before_any_launch(lib):
    f, need = lib.sandwich_norm_backward, lib.sandwich_norm_backward_workspace_size
    a, b, c, d, e = (ctypes.c_void_p(1 << (20 + i)) for i in range(5))
    tail = (1.0, 1.0, a, b, P, P, N, P, need(4, 64), N)
    assert f(c, 5, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 64, *tail) == -1
    assert f(c, 0, d, e, 0, P, P, P, 0, N, N, N, 0, 4, 64, *tail) == -1       # dy without w_next
    assert f(c, 0, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 40, *tail) == -2
    assert f(c, 0, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 64, 1.0, 1.0, a, b, P, P, P, P, need(4, 64), N) == -1   # dgate without gate
    assert f(c, 0, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 64, 1.0, 1.0, a, b, N, P, N, P, need(4, 64), N) == -1   # dw_next without dw_post
    assert f(c, 0, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 64, 1.0, 1.0, a, b, P, P, N, P, need(4, 64) - 1, N) == -3
    assert f(N, 0, N, e, 0, P, P, P, 0, N, N, N, 0, 4, 64, 1.0, 1.0, a, b, P, N, N, P, need(4, 64), N) == -1   # no gradient at all
    assert f(c, 0, d, e, 0, P, P, P, 0, P, P, N, 0, 4, 64, 1.0, 1.0, a, a, P, P, N, P, need(4, 64), N) == -1   # dx is dresidual
    assert b"overlaps" in lib.invmoe_last_error()
    assert need(0, 64) == 256
    assert need(2 ** 31 - 1, 64) > 2 ** 33                                      # counted without wrapping


def test_verify_drafts_rejects_before_any_launch(lib):
    f, need = lib.verify_drafts, lib.verify_workspace_size
    out = (P, P, P)
    ok = need(2, 3, 100)
    assert f(P, 9, N, P, P, P, N, N, 1.0, 2, 3, 100, *out, P, ok, N) == -1
    assert f(P, 1, N, P, P, P, N, N, -0.5, 2, 3, 100, *out, P, ok, N) == -1
    assert f(P, 1, N, P, P, P, N, N, 1.0, 2, 33, 100, *out, P, 1 << 30, N) == -2
    assert f(P, 1, N, P, P, P, N, N, 1.0, 2, 3, 0, *out, P, ok, N) == -1
    assert f(P, 1, N, P, P, P, N, N, 1.0, 2, 3, 100, *out, P, ok - 1, N) == -3
    assert f(P, 1, N, N, P, P, N, N, 1.0, 2, 3, 100, *out, P, ok, N) == -1 and b"draft_tokens" in lib.invmoe_last_error()
    assert f(P, 1, P, N, N, P, N, N, 1.0, 2, 0, 100, *out, P, ok, N) == -1
    assert f(ctypes.c_void_p(4097), 1, N, P, P, P, N, N, 1.0, 2, 3, 100, *out, P, ok, N) == -4
    assert f(P, 1, N, P, P, P, N, N, 1.0, 2 ** 31 - 1, 3, 151552, *out, P, 2 ** 62, N) == -2
    assert f(P, 1, N, P, P, P, N, N, 1.0, 0, 3, 100, *out, P, ok, N) == 0
    assert need(0, 3, 100) == 256 and need(2 ** 31 - 1, 32, 2 ** 31 - 1) > 2 ** 45


def test_moe_layer_decode_rejects_before_any_launch(lib):
    f, need = lib.moe_layer_decode, lib.moe_decode_workspace_size
    x, o, b, ws = (ctypes.c_void_p(1 << (20 + i)) for i in range(4))

    def call(T=4, H=256, E=8, k=2, F=128, Fs=0, score=2, bias=N, groups=1, kept=1, renorm=1, scale=1.0, x=x, out=o, n=None):
        n = need(T, H, E, k, F, Fs) if n is None else n
        return f(x, P, P, P, N, N, T, H, E, k, F, Fs, score, bias, groups, kept, renorm, scale, out, N, N, N, N, ws, n, N)
    assert call(T=17, n=1 << 30) == -2 and b"T=17" in lib.invmoe_last_error()
    assert call(E=513) == -2 and call(H=100) == -2 and call(F=96) == -2 and call(Fs=32) == -2 and call(H=32832) == -2
    assert call(k=9) == -1 and call(E=64, k=33) == -2 and call(T=-1) == -1
    assert call(score=3) == -1 and call(bias=b) == -1 and call(scale=2.0) == -1 and call(renorm=0) == -1
    assert call(score=0, groups=3) == -1 and call(score=0, groups=4, kept=5) == -1 and call(score=0, groups=8, kept=1) == -1
    assert call(n=need(4, 256, 8, 2, 128, 0) - 1) == -3
    assert call(out=N) == -1 and call(Fs=64) == -1                    # no output; no shared weights
    assert call(x=ctypes.c_void_p(4100)) == -4
    assert call(x=o) == -1 and b"overlaps" in lib.invmoe_last_error()
    assert call(T=0) == 0
    assert need(17, 256, 8, 2, 128, 0) == 256 and need(16, 32768, 512, 32, 1 << 20, 1 << 20) > 2 ** 30


def test_binding_refuses_host_tensors():
    from serve_invariant_moe_gb300 import binding
    x, w = torch.zeros(4, 64), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.sandwich_norm(x, w, x, w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.sandwich_norm_backward(x, x, x, w, torch.zeros(4), x, w, torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.verify_drafts(torch.zeros(2, 1, 8), torch.zeros(2, 8), torch.zeros(256, dtype=torch.uint8))
    h = w.view(1, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.moe_layer_decode(h, h, h.view(1, 1, 64).expand(1, 2, 64), h.view(1, 64, 1), 1, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="2 dimensions"):
        binding.sandwich_norm(x[0], w, x, w)
    with pytest.raises(ValueError, match="3 dimensions"):
        binding.verify_drafts(torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(256, dtype=torch.uint8))


def test_verify_drafts_rejects_columns_past_its_index(lib):
    """A chunk past the last column of a row has to have an index too."""
    f = lib.verify_drafts
    for V in (2 ** 30 + 1, 2 ** 31 - 4, 2 ** 31 - 1):
        assert f(P, 1, N, N, N, P, N, N, 1.0, 1, 0, V, P, P, P, P, 2 ** 62, N) == -2 and b"2^30" in lib.invmoe_last_error()


def test_moe_layer_decode_rejects_outputs_that_overlap(lib):
    f, n = lib.moe_layer_decode, lib.moe_decode_workspace_size(4, 256, 8, 2, 128, 0)
    at = [(1 << 20) + (i << 16) for i in range(6)]                   # x, out, out_bf16, logits, topk_idx, topk_w
    size = [4 * 256 * 2, 4 * 256 * 4, 4 * 256 * 2, 4 * 8 * 4, 4 * 2 * 4, 4 * 2 * 4]
    for i in range(6):
        for j in range(i):
            p = [ctypes.c_void_p(a) for a in at]
            p[i] = ctypes.c_void_p(at[j] + size[j] - 16)             # its first bytes are the other's last
            assert f(p[0], P, P, P, N, N, 4, 256, 8, 2, 128, 0, 2, N, 1, 1, 1, 1.0, *p[1:], ctypes.c_void_p(1 << 24), n, N) == -1
            assert b"overlaps" in lib.invmoe_last_error(), (i, j)


class FakeLayerBinding:
    """The binding's functions that MoELayer's decode calls; the workspace of `fail` is one whose kernel gave up a wait."""
    DECODE_MAX_TOKENS, DECODE_MAX_EXPERTS = 16, 512

    def plan_len(self, T, E, k):
        return 2 * E + 1 + 2 * T * k

    def workspace_size(self, T, *more):
        return 256 + 64 * T

    moe_decode_workspace_size = workspace_size

    def new_workspace(self, nbytes, device):
        return torch.zeros(nbytes, dtype=torch.uint8)

    def check_status(self, workspace):
        if workspace[0]:
            workspace[0] = 0
            raise RuntimeError("timeout")

    def lib(self):
        return types.SimpleNamespace(moe_layer_forward=lambda *args: 0)

    def check(self, rc):
        assert rc == 0

    def moe_layer_decode(self, x, w_router, w13, w2, k, workspace, *more, out=None, **rest):
        return dict(out=out)

    def moe_layer_forward(self, x, w_router, w13, w2, k, ws, **rest):
        return dict(out=None)


@pytest.fixture
def layer(monkeypatch):
    from serve_invariant_moe_gb300 import api
    monkeypatch.setattr(api, "binding", FakeLayerBinding())
    stream = types.SimpleNamespace(wait_stream=lambda other: None, cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "Stream", lambda **kw: stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "graph", lambda g: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: types.SimpleNamespace(replay=lambda: None))
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16)   # noqa: E731
    return api.MoELayer(api.MoEWeights(bf16(4, 64), bf16(4, 256, 64), bf16(4, 64, 128), 2), fused=True)


def rows(T):
    return torch.empty(T, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("name", ["ws", "fused_ws"])
def test_check_covers_replaced_decode_buffers(layer, name):
    layer.check()
    layer.decode(rows(2))
    layer._decode[name][0] = 1
    layer.decode(rows(9))                           # larger buffers
    with pytest.raises(RuntimeError, match="timeout"):
        layer.check()
    layer.check()


def test_check_covers_prefill(layer):
    for replaced in (False, True):
        layer.prefill(rows(8), return_all=True)
        layer._ws[0] = 1
        if replaced:
            layer.prefill(rows(2000))
        with pytest.raises(RuntimeError, match="timeout"):
            layer.check()
        layer.check()


@pytest.mark.parametrize("name", ["ws", "fused_ws"])
def test_check_covers_decode_graphs(layer, name):
    from serve_invariant_moe_gb300 import api
    graphs = api.DecodeGraphs(layer, buckets=(1, 4))
    layer.decode(rows(9))
    graphs.check()
    graphs._bufs[name][0] = 1                       # what a replayed kernel does
    layer.check()
    with pytest.raises(RuntimeError, match="timeout"):
        graphs.check()
    graphs.check()


def test_the_blocks_backward_checks_its_norms(monkeypatch):
    from serve_invariant_moe_gb300 import block

    class Fake(FakeLayerBinding):
        def sandwich_norm_backward_workspace_size(self, T, H):
            return 256 + T * H

        def sandwich_norm_backward(self, *args, workspace, **rest):
            workspace[0] = self.fail
            return dict(dx=None, dresidual=None, dw_post=None, dw_next=None, dgate=None)
    fake = Fake()
    monkeypatch.setattr(block, "binding", fake)
    w = torch.ones(64, dtype=torch.bfloat16)
    b = object.__new__(block.MoEBlock)
    b.w, b._norm_ws = block.MoEBlockWeights(None, w, w), None
    b.layer = types.SimpleNamespace(backward=lambda *args: dict(dx=None))
    fwd = dict(layer=dict(out=None), rstd_post=None, residual=rows(3), rstd=None, gate=None, n=None)
    fake.fail = 0
    b.backward(fwd, rows(3))
    fake.fail = 1
    with pytest.raises(RuntimeError, match="timeout"):
        b.backward(fwd, rows(3))


@pytest.fixture
def capture(monkeypatch):
    """capture(True): the calls from here on are captured."""
    now = [False]
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0])
    return lambda on: now.__setitem__(0, on)


def memory(buffers):
    return {name: weakref.ref(t) for name, t in buffers.items() if isinstance(t, torch.Tensor)}


@pytest.mark.parametrize("fused", [True, False])
def test_a_caller_s_graph_keeps_the_buffers_of_its_step(layer, capture, fused):
    """A larger batch gives the layer new buffers; the kernels that a caller captured still write the old ones."""
    layer.fused = fused
    layer.decode(rows(2))
    capture(True)
    layer.decode(rows(2))
    capture(False)
    used = memory(layer._decode)
    assert {"logits", "plan", "xp", "h", "y", "out", "ws"} <= set(used)
    layer.decode(rows(9))
    gc.collect()
    assert [name for name, r in used.items() if r() is None] == []
    unused = memory(layer._decode)
    layer.decode(rows(30))
    gc.collect()
    assert all(r() is None for r in unused.values())        # (nobody captured these)
    used["ws"]()[0] = 1                                     # what a replayed kernel does
    with pytest.raises(RuntimeError, match="timeout"):
        layer.check()
    layer.check()


def test_a_captured_first_step_has_buffers_of_its_own(layer, capture):
    """Inside a capture nothing is cleared before the first replay: an eager step must not find those workspaces."""
    capture(True)
    layer.decode(rows(2))
    assert layer._decode is None
    with pytest.raises(RuntimeError, match="captured"):
        layer.alloc_decode(4)
    capture(False)
    layer.decode(rows(2))
    kept = memory(layer._captured[0])
    assert layer._decode["ws"] is not kept["ws"]() and kept["ws"]() is not None
    kept["ws"]()[0] = 1
    with pytest.raises(RuntimeError, match="timeout"):
        layer.check()


def test_a_captured_prefill_has_a_workspace_of_its_own(layer, capture):
    layer.prefill(rows(8), return_all=True)
    eager = layer._ws
    capture(True)
    layer.prefill(rows(8), return_all=True)
    capture(False)
    assert layer._ws is eager and layer._captured[0]["ws"] is not eager


class Recorder(FakeLayerBinding):
    """Remembers the workspace and the logits' buffer of every call."""

    def __init__(self):
        self.seen = []

    def moe_layer_decode(self, x, w_router, w13, w2, k, workspace, *more, logits, **rest):
        self.seen.append((workspace, logits.untyped_storage().data_ptr()))
        return dict(out=None)

    def moe_layer_forward(self, x, w_router, w13, w2, k, ws, logits=None, **rest):
        self.seen.append((ws, None if logits is None else logits.untyped_storage().data_ptr()))
        return dict(out=None)

    def check_status(self, workspace):
        self.seen.append((workspace, None))

    backward_workspace_size = FakeLayerBinding.workspace_size

    def gradients(self, *args, **kw):
        return collections.defaultdict(lambda: None)

    moe_combine_backward = moe_grouped_ffn_backward = moe_route_backward = gradients


CALLS = {"fused": lambda layer: layer.prefill(rows(8)), "small": lambda layer: layer.prefill(rows(100)),
         "all": lambda layer: layer.prefill(rows(8), return_all=True), "large": lambda layer: layer.prefill(rows(2000)),
         "backward": lambda layer: layer.backward(rows(8), collections.defaultdict(lambda: None), None)}


@pytest.mark.parametrize("call", CALLS)
def test_prefills_and_backwards_of_two_callers_share_nothing(layer, capture, monkeypatch, call):
    """Two threads or streams whose calls overlap: neither the workspace nor the logits that every block chooses from."""
    from serve_invariant_moe_gb300 import api
    rec, stream = Recorder(), [0]
    monkeypatch.setattr(api, "binding", rec)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: stream[0], raising=False)
    for stream[0] in (5, 6, 5):
        CALLS[call](layer)
    t = threading.Thread(target=CALLS[call], args=(layer,))
    t.start()
    t.join()
    layer.decode(rows(8))
    (a, la), (b, lb), (again, lagain), (c, lc), (d, ld) = (*rec.seen, (None, None))[:5]
    assert again is a and lagain == la
    assert len({id(s) for s in (a, b, c, d)}) == 4
    assert la is None or len({la, lb, lc, ld}) == 4


def test_two_backwards_of_a_block_share_no_partial_sums(monkeypatch):
    """Two threads: the second call's row kernel may run before the first one's sum kernel."""
    from serve_invariant_moe_gb300 import block
    spaces = []

    class Fake(FakeLayerBinding):
        def sandwich_norm_backward_workspace_size(self, T, H):
            return 256 + T * H

        def sandwich_norm_backward(self, *args, workspace, **rest):
            assert workspace.numel() >= 256 + 3 * 64 and not workspace[:256].any()
            spaces.append(workspace)
            if len(spaces) == 1:                    # the other thread's call, before this one is done
                t = threading.Thread(target=b.backward, args=(fwd, rows(3)))
                t.start()
                t.join()
            return dict(dx=None, dresidual=None, dw_post=None, dw_next=None, dgate=None)
    monkeypatch.setattr(block, "binding", Fake())
    w = torch.ones(64, dtype=torch.bfloat16)
    b = object.__new__(block.MoEBlock)
    b.w, b._norm_ws = block.MoEBlockWeights(None, w, w), None
    b.layer = types.SimpleNamespace(backward=lambda *args: dict(dx=None))
    fwd = dict(layer=dict(out=None), rstd_post=None, residual=rows(3), rstd=None, gate=None, n=None)
    b.backward(fwd, rows(3))
    assert len(spaces) == 2 and spaces[0].data_ptr() != spaces[1].data_ptr()


def test_the_stalled_backward_rejects_before_any_launch(lib):
    f, need = lib.invmoe_debug_stalled_backward, lib.sandwich_norm_backward_workspace_size
    a, b = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)

    def call(T=4, H=64, group=0, us=1000, dy=P, n=None):
        return f(dy, P, P, P, P, P, P, P, T, H, group, us, a, b, P, P, P, need(T, H) if n is None else n, N)
    assert call(T=0) == -2 and call(H=2064) == -2 and call(group=2) == -1 and call(us=0) == -1 and call(us=2000001) == -1
    assert call(dy=N) == -1 and call(dy=ctypes.c_void_p(4100)) == -4 and call(n=need(4, 64) - 1) == -3


@pytest.mark.parametrize("given", [False, True])
def test_the_head_s_time_out_can_be_read_without_a_workspace_of_the_caller_s(monkeypatch, given):
    from serve_invariant_moe_gb300 import api

    class Fake(FakeLayerBinding):
        def workspace_size(self, T, H, V):
            return 512

        def verify_workspace_size(self, B, D, V):
            return 1024

        def lm_logprob_kl(self, hidden, w_vocab, target, workspace, logits, write_logits):
            assert workspace.numel() >= 1024 and not workspace[:256].any()
            workspace[0] = 1                        # what a kernel that gives up does
            return dict(logits=torch.zeros(hidden.shape[0], w_vocab.shape[0]))

        def verify_drafts(self, z, noise, workspace, *more):
            return dict(tokens=None)
    fake = Fake()
    monkeypatch.setattr(api, "binding", fake)
    ws = torch.zeros(1024, dtype=torch.uint8) if given else None
    got = api.head_verify_drafts(rows(3), torch.empty(16, 64), torch.ones(3, 16), workspace=ws)
    assert ("workspace" in got) is not given
    with pytest.raises(RuntimeError, match="timeout"):
        fake.check_status(ws if given else got["workspace"])


def layer_of(E, H, F=64, Fs=0):
    """Weights of a size, without their memory."""
    from serve_invariant_moe_gb300 import api
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="meta")   # noqa: E731
    return api.MoEWeights(e(E, H), e(E, 2 * F, H), e(E, H, F), 2, e(2 * Fs, H) if Fs else None, e(H, Fs) if Fs else None)


@pytest.mark.parametrize("size,fits", [((512, 64), True), ((600, 64), False), ((4, 32768), True), ((4, 32832), False),
                                       ((4, 64, (1 << 20) + 64), False), ((4, 64, 64, (1 << 20) + 64), False)])
def test_the_one_kernel_layer_is_taken_where_it_fits(size, fits):
    """A block of any layer can be built, and whether few rows go through one kernel is known from the start."""
    from serve_invariant_moe_gb300 import api, block
    w = layer_of(*size)
    assert api.MoELayer(w).fused is False and api.MoELayer(w, fused=None).fused is fits
    assert block.MoEBlock(block.MoEBlockWeights(w, None)).layer.fused is fits
    if fits:
        assert api.MoELayer(w, fused=True).fused
    else:
        with pytest.raises(ValueError, match="fused"):
            api.MoELayer(w, fused=True)
        with pytest.raises(ValueError, match="fused"):
            block.MoEBlock(block.MoEBlockWeights(w, None), fused=True)


def test_verify_drafts_rejects_outputs_that_overlap(lib):
    """Tokens over the drafted ones, say: a request's would be written while the next one's drafts are read."""
    f, B, D, V = lib.verify_drafts, 3, 2, 96
    n = lib.verify_workspace_size(B, D, V)
    # logits, draft_logits, draft_tokens, accept_u, noise, n_draft, temperature, tokens, n_accepted, logp
    size = [B * (D + 1) * V * 4, B * D * V * 4, B * D * 4, B * D * 4, B * V * 4, B * 4, B * 4, B * (D + 1) * 4, B * 4, B * (D + 1) * 4]
    at = [(1 << 20) + (i << 16) for i in range(10)]
    for i in (7, 8, 9):
        for j in range(i):
            for first in (at[j], at[j] + size[j] - 4, at[j] - size[i] + 4):
                p = [ctypes.c_void_p(a) for a in at]
                p[i] = ctypes.c_void_p(first)
                assert f(p[0], 1, *p[1:7], 1.0, B, D, V, *p[7:], ctypes.c_void_p(1 << 24), n, N) == -1, (i, j)
                assert b"overlaps" in lib.invmoe_last_error(), (i, j)


def overlapping(size, outs):
    """Addresses of arrays that lie apart, with output i moved onto array j: on it, over its end, over its begin."""
    at = [(1 << 20) + (i << 16) for i in range(len(size))]
    for i in outs:
        for j in range(len(size)):
            if i != j:
                for first in (at[j], at[j] + size[j] - 16, at[j] - size[i] + 16):
                    yield i, j, first - at[j], [ctypes.c_void_p(first if k == i else a) for k, a in enumerate(at)]


@pytest.mark.parametrize("kind", [1, 2])
def test_sandwich_norm_rejects_every_overlap(lib, kind):
    """Also of the rows' numbers with the weights, the gate or one another; residual_out alone may be the residual."""
    T, H = 4, 64
    row, small = T * H, T * 4
    # x, w_post, residual, gate, w_next, residual_out, out, q, scale, rstd_post, rstd
    size = [row * 4, H * 2, row * 2, H * 2 if kind == 1 else small, H * 2, row * 2, row * 2, row, small, small, small]
    for i, j, shift, p in overlapping(size, range(5, 11)):
        if (i, j, shift) == (5, 2, 0):
            continue
        rc = lib.sandwich_norm(p[0], 1, p[1], p[2], 0, p[3], kind, p[4], T, H, 1.0, 1.0, 1e-6, *p[5:], N)
        assert rc in (-1, -4) and (rc == -4 or b"overlaps" in lib.invmoe_last_error()), (i, j, shift)


@pytest.mark.parametrize("kind", [1, 2])
def test_sandwich_norm_backward_rejects_every_overlap(lib, kind):
    T, H = 4, 64
    row, small = T * H, T * 4
    # dy, dres, x, w_post, rstd_post, residual, w_next, rstd, gate, dx, dresidual, dw_post, dw_next, dgate
    size = [row * 2, row * 2, row * 4, H * 2, small, row * 2, H * 2, small, H * 2 if kind == 1 else small, row * 4, row * 2,
            H * 4, H * 4, H * 4 if kind == 1 else small]
    n = lib.sandwich_norm_backward_workspace_size(T, H)
    for i, j, shift, p in overlapping(size, range(9, 14)):
        rc = lib.sandwich_norm_backward(p[0], 0, p[1], p[2], 1, p[3], p[4], p[5], 0, p[6], p[7], p[8], kind, T, H, 1.0, 1.0,
                                        *p[9:], ctypes.c_void_p(1 << 24), n, N)
        assert rc in (-1, -4) and (rc == -4 or b"overlaps" in lib.invmoe_last_error()), (i, j, shift)


def test_moe_layer_decode_wants_both_weights_of_the_shared_expert():
    from serve_invariant_moe_gb300 import binding
    e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)   # noqa: E731
    for shared in (dict(ws2=e(64, 64)), dict(ws13=e(128, 64))):
        with pytest.raises(ValueError, match="ws13 and ws2"):
            binding.moe_layer_decode(e(2, 64), e(4, 64), e(4, 128, 64), e(4, 64, 64), 1, torch.zeros(256, dtype=torch.uint8), **shared)
