"""Host side of the 8-bit block and of the decode graphs on CPU: what the objects keep alive and which status words the
block's check reads.

The library's calls are replaced by fakes on CPU tensors, CUDA graphs and streams by objects that do nothing."""
import contextlib
import gc
import threading
import types
import weakref

import pytest
import torch

from serve_invariant_moe_gb300 import api, block


class FakeBinding:
    """The binding's functions that the block calls; `fail` names one whose kernel gives up a wait."""
    FP8 = torch.float8_e4m3fn

    def __init__(self):
        self.fail = None
        self.stream = 0

    def _call(self, name, workspace):
        if name == self.fail:
            workspace[0] = 1

    def plan_len(self, T, E, k):
        return 2 * E + 1 + 2 * T * k

    def workspace_size(self, T, H, E, k, *more):
        return 256 + 4 * T * E

    def new_workspace(self, nbytes, device):
        return torch.zeros(max(nbytes, 256), dtype=torch.uint8)

    def check_status(self, workspace):
        if workspace[0]:
            workspace[0] = 0
            raise RuntimeError("timeout")

    def _stream(self):
        return self.stream

    def add_rms_norm(self, x, w, residual, eps, out, fp8, residual_out, q, scale, rstd):
        if residual is not None and residual_out is not None:
            n = residual.numel() * residual.element_size()
            apart = abs(residual.data_ptr() - residual_out.data_ptr())
            assert apart == 0 or apart >= n, "rows that one block writes are read by another"
            residual_out.copy_(residual)
        return dict(out=out, q=q, scale=scale, rstd=rstd, residual=residual_out)

    def moe_router_logits(self, x, w, ws, logits):
        self._call("moe_router_logits", ws)
        return logits

    def moe_route_select(self, logits, k, score, bias, n_group, topk_group, renormalize, scale, idx, w, plan, ws):
        assert ws.numel() >= self.workspace_size(logits.shape[0], 0, logits.shape[1], k)
        return dict(topk_idx=idx, topk_w=w, plan=plan)

    def moe_permute_fp8(self, q, scale, plan, E, k, xp, xs):
        return xp, xs

    def moe_grouped_swiglu_fp8(self, xp, xs, plan, w13, s13, T, k, ws, h, hs):
        self._call("moe_grouped_swiglu_fp8", ws)
        return dict(h=h, h_scale=hs)

    def moe_grouped_down_fp8(self, h, hs, plan, w2, s2, T, k, ws, y):
        self._call("moe_grouped_down_fp8", ws)
        return y

    def lib(self):
        return types.SimpleNamespace(moe_layer_forward=lambda *args: 0)

    def check(self, rc):
        assert rc == 0

    def moe_combine(self, y, w, plan, T, H, E, k, y_shared, out, out_bf16):
        return torch.zeros(T, H) if out is None else out


@pytest.fixture
def fake(monkeypatch):
    f = FakeBinding()
    monkeypatch.setattr(block, "binding", f)
    monkeypatch.setattr(api, "binding", f)
    stream = types.SimpleNamespace(wait_stream=lambda other: None, cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "Stream", lambda **kw: stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "graph", lambda g: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "CUDAGraph", lambda: types.SimpleNamespace(replay=lambda: None))
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return f


def weights(E=4, H=128, F=128, Fs=128):
    e = lambda *s, dtype=torch.float8_e4m3fn: torch.empty(*s, dtype=dtype)   # noqa: E731
    f = lambda *s: torch.empty(*s)                                           # noqa: E731
    bf16 = torch.bfloat16
    return block.Fp8MoEWeights(e(H, dtype=bf16), e(E, H, dtype=bf16), e(E, 2 * F, H), f(E, 2 * F // 128, H // 128),
                               e(E, H, F), f(E, H // 128, F // 128), 2, api.Routing(bias=f(E)), e(1, 2 * Fs, H),
                               f(1, 2 * Fs // 128, H // 128), e(1, H, Fs), f(1, H // 128, Fs // 128))


def memory(w):
    """A weak reference to the memory of every tensor that a step reads."""
    tensors = [t for t in [*vars(w).values(), w.routing.bias] if isinstance(t, torch.Tensor)]
    assert len(tensors) == 11
    return [weakref.ref(t) for t in tensors]


def test_a_graph_keeps_what_its_kernels_read(fake):
    """Captured kernels hold addresses: the weights must outlive the caller's last reference to the block."""
    w = weights()
    refs = memory(w)
    g = block.Fp8DecodeGraph(block.Fp8MoEBlock(w), 3)
    del w
    gc.collect()
    assert all(r() is not None for r in refs)
    del g
    gc.collect()
    assert all(r() is None for r in refs)


def test_a_graph_keeps_what_its_kernels_read_when_the_weights_are_exchanged(fake):
    w = weights()
    refs = memory(w)
    b = block.Fp8MoEBlock(w)
    g = block.Fp8DecodeGraph(b, 3)
    new = weights()
    for name, t in vars(new).items():
        setattr(w, name, t)
    gc.collect()
    assert all(r() is not None for r in refs)
    del g
    gc.collect()
    assert all(r() is None for r in refs)


def test_decode_graphs_keep_their_buffers_and_weights(fake):
    """A larger batch, decoded or prefilled, gives the layer new buffers; the captured steps still write the old ones."""
    bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16)   # noqa: E731
    w = api.MoEWeights(bf16(4, 64), bf16(4, 256, 64), bf16(4, 64, 128), 2)
    layer = api.MoELayer(w)
    graphs = api.DecodeGraphs(layer, buckets=(1, 4))
    buffers = {name: weakref.ref(t) for name, t in layer._decode.items() if isinstance(t, torch.Tensor)}
    read = [weakref.ref(t) for t in (w.w_router, w.w13, w.w2)]
    assert {"logits", "plan", "xp", "h", "y", "out", "ws"} <= set(buffers)
    layer.decode(bf16(9, 64))
    w.w_router, w.w13, w.w2 = bf16(4, 64), bf16(4, 256, 64), bf16(4, 64, 128)
    gc.collect()
    assert [name for name, r in buffers.items() if r() is None] == []
    assert all(r() is not None for r in read)
    del graphs
    gc.collect()
    assert all(r() is None for r in [*buffers.values(), *read])


FAILING = ["moe_router_logits", "moe_grouped_swiglu_fp8", "moe_grouped_down_fp8"]


@pytest.mark.parametrize("fail", FAILING)
def test_check_covers_prefill(fake, fail):
    """On every stream, also of calls before a larger batch, and each time-out is reported once."""
    b = block.Fp8MoEBlock(weights())
    b.check()
    for stream, T in [(0, 8), (1, 3), (0, 3)]:
        fake.stream, fake.fail = stream, fail
        b.prefill(torch.empty(T, 128))
        fake.fail = None
        b.prefill(torch.empty(5 * T, 128))          # needs a larger workspace
        with pytest.raises(RuntimeError, match="timeout"):
            b.check()
        b.check()


def test_streams_and_threads_do_not_share_a_workspace(fake):
    b = block.Fp8MoEBlock(weights())
    spaces = []

    def run():
        spaces.append(b.prefill(torch.empty(4, 128), return_all=True)["workspace"])
    for stream in (0, 1, 0):
        fake.stream = stream
        run()
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert spaces[0] is spaces[2] and spaces[0] is not spaces[1] and spaces[3] is not spaces[0]


@pytest.mark.parametrize("fail", FAILING)
def test_check_covers_replaced_decode_buffers(fake, fail):
    b = block.Fp8MoEBlock(weights())
    x, res = torch.empty(9, 128), torch.empty(9, 128, dtype=torch.bfloat16)
    fake.fail = fail
    b.decode(x[:2], res[:2])
    fake.fail = None
    b.decode(x, res)
    with pytest.raises(RuntimeError, match="timeout"):
        b.check()
    b.check()


@pytest.mark.parametrize("fail", FAILING)
def test_check_covers_graphs(fake, fail):
    b = block.Fp8MoEBlock(weights())
    g = block.Fp8DecodeGraph(b, 2)
    g.check()
    fake.fail = fail
    fake._call(fail, g._bufs["ws"])                 # what a replayed kernel does
    with pytest.raises(RuntimeError, match="timeout"):
        g.check()
    g.check()


def test_check_covers_a_prefill_that_a_caller_captures(fake, monkeypatch):
    """Its workspace belongs to the captured graph: no other call uses it, and every replay's status is read."""
    b = block.Fp8MoEBlock(weights())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    ws = b.prefill(torch.empty(4, 128), return_all=True)["workspace"]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    assert b.prefill(torch.empty(4, 128), return_all=True)["workspace"] is not ws
    for _ in range(2):
        ws[0] = 1
        with pytest.raises(RuntimeError, match="timeout"):
            b.check()
        b.check()


def test_decode_of_some_of_the_last_step_s_requests(fake):
    """Rows of the returned residual are a view of the buffer that the next step writes: shifted ones are read first."""
    b = block.Fp8MoEBlock(weights())
    x, res = torch.empty(6, 128), torch.arange(6 * 128).view(6, 128).to(torch.bfloat16)
    _, r = b.decode(x, res)
    _, same = b.decode(x, r)
    assert same.data_ptr() == r.data_ptr() and torch.equal(same, res)
    _, r = b.decode(x[1:4], r[1:4])
    assert torch.equal(r, res[1:4])
    _, r = b.decode(x[2:3], r[2:])
    assert torch.equal(r, res[3:4])


def test_the_norm_refuses_partly_overlapping_rows():
    """Before anything is launched: the addresses are never read."""
    import ctypes
    from serve_invariant_moe_gb300 import _lib, build
    build.build()
    lib, p, null = _lib.lib(), ctypes.c_void_p, None
    T, H, at = 3, 64, 1 << 20
    for shift in (-T * H * 2 + 16, -128, 16, 128, T * H * 2 - 16):
        assert lib.add_rms_norm(p(4096), 0, p(at), 0, p(8192), T, H, 1e-6, p(at + shift), p(16384), null, null, null,
                                null) == -1
        assert b"overlaps" in lib.invmoe_last_error()
        assert lib.add_rms_norm_backward(p(4096), 0, p(8192), 0, p(8192), p(8192), p(at), T, H, p(at + shift), null, null,
                                         0, null) == -1
        assert b"overlaps" in lib.invmoe_last_error()
