"""Prefill and decode entry points over the C ABI.

Both entry points run the same three library calls (moe_route_topk,
moe_grouped_ffn, moe_combine) with the same kernels and tile shapes; they differ
only on the host side.  Prefill takes any number of tokens in one call; decode
serves one token per request from buffers allocated once for a maximum batch.
Because every reduction in the library is per token with a fixed order, a
token's output bits do not depend on which entry point served it or on what
else was in its batch ("位级一致：前沿训练的差异化关键", section "端到端零 KLD":
the serving engine and the trainer must produce the same numbers whatever the
batch size or concurrent load).
"""
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding


@dataclass
class Routing:
    """Expert choice by scores (binding.moe_route_select); without one a layer's router is the softmax over its top-k logits."""
    score: str = "sigmoid"                # or "softmax"
    bias: Optional[torch.Tensor] = None   # [E] fp32, added to the scores for the choice alone
    n_group: int = 1
    topk_group: int = 1
    renormalize: bool = True
    scale: float = 1.0

    def select(self, logits, k, workspace, topk_idx=None, topk_w=None, plan=True):
        return binding.moe_route_select(logits, k, self.score, self.bias, self.n_group, self.topk_group,
                                        self.renormalize, self.scale, topk_idx, topk_w, plan, workspace)


@dataclass
class MoEWeights:
    w_router: torch.Tensor            # [E, H] bf16
    w13: torch.Tensor                 # [E, 2F, H] bf16 (gate rows, then up rows)
    w2: torch.Tensor                  # [E, H, F] bf16
    k: int
    ws13: Optional[torch.Tensor] = None   # [2Fs, H] bf16 shared expert
    ws2: Optional[torch.Tensor] = None    # [H, Fs] bf16
    routing: Optional[Routing] = None

    @property
    def E(self):
        return self.w13.shape[0]

    @property
    def H(self):
        return self.w13.shape[2]

    @property
    def F(self):
        return self.w13.shape[1] // 2

    @property
    def F_shared(self):
        return 0 if self.ws13 is None else self.ws13.shape[0] // 2


def _head(t, n):
    """The first n rows of a buffer that may be absent."""
    return None if t is None else t[:n]


def _capturing():
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _caller():
    """The calling thread and its current stream: calls with the same ones run one after the other.  None in a capture."""
    if not torch.cuda.is_initialized():
        return threading.get_ident(), 0
    if torch.cuda.is_current_stream_capturing():
        return None
    return threading.get_ident(), torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


FUSED_MAX_WIDTH = 32768                  # of the one-kernel layer's rows


def fused_fits(w: MoEWeights) -> bool:
    """Whether the one-kernel layer (binding.moe_layer_decode) takes these weights."""
    return w.E <= binding.DECODE_MAX_EXPERTS and w.H <= FUSED_MAX_WIDTH and max(w.F, w.F_shared) <= 1 << 20


def _overlap(a, b):
    """Two contiguous tensors have a byte in common."""
    x, y = a.data_ptr(), b.data_ptr()
    return x < y + b.numel() * b.element_size() and y < x + a.numel() * a.element_size()


def _check_all(spaces):
    """check_status of every workspace, so that each time-out is reported once."""
    failed = None
    for ws in spaces:
        try:
            binding.check_status(ws)
        except RuntimeError as e:
            failed = e
    if failed is not None:
        raise failed


class MoELayer:
    """Batch-invariant MoE layer forward on one GPU.

    fused: decode (and prefill without its intermediates) of at most 16 tokens runs the layer in one kernel
    (binding.moe_layer_decode, at most 512 experts and 32768 columns), with the same bits; the decode buffers of its
    intermediates (xp, h, y, ys, plan) are then not written.  An out_bf16 that overlaps the tokens takes the separate kernels.
    None: where the weights fit.

    prefill and backward may run on several threads and streams at once: each has workspaces of its own there.  The calls of
    decode share one set of buffers, so they belong on one stream.

    Captured kernels hold addresses: the buffers that a captured call uses live as long as the layer, also when a larger batch
    gives it others, so a caller's own graph needs the layer (and its weights) kept.  DecodeGraphs keeps its buffers itself."""

    def __init__(self, weights: MoEWeights, fused: Optional[bool] = False):
        fits = (fused is None or bool(fused)) and fused_fits(weights)
        if fused and not fits:
            raise ValueError(f"fused decode takes at most {binding.DECODE_MAX_EXPERTS} experts and {FUSED_MAX_WIDTH} columns, "
                             f"got {weights.E} and {weights.H} (F {weights.F}, shared {weights.F_shared})")
        self.w = weights
        self.fused = fits
        self._spaces, self._small, self._back = {}, {}, {}      # prefill's and backward's, by thread and stream
        self._decode = None
        self._unread = []               # status blocks of replaced workspaces, which check() reads
        self._captured = []             # buffers that a caller's graphs use

    @property
    def _ws(self):
        """prefill's workspace of this thread on the current stream."""
        return self._spaces.get(_caller())

    def _workspace(self, T):
        w = self.w
        return self._kept(self._spaces, binding.workspace_size(T, w.H, w.E, w.k, w.F, w.F_shared, 0))

    def _kept(self, spaces, need):
        """The caller's workspace in `spaces`, of at least `need` bytes; a captured call's is its graph's."""
        key = _caller()
        if key is None:
            self._captured.append(dict(ws=binding.new_workspace(need, self.w.w13.device)))
            return self._captured[-1]["ws"]
        ws = spaces.get(key)
        if ws is None or ws.numel() < need:
            self._replace(ws)
            ws = spaces[key] = binding.new_workspace(need, device=self.w.w13.device)
        return ws

    def _run(self, x, ws, bufs=None, out_bf16=None, replay_idx=None):
        w = self.w
        T = x.shape[0]
        bufs = bufs or {}
        if w.routing is not None:
            return self._run_routed(x, ws, bufs, out_bf16, replay_idx)
        if replay_idx is None:
            # route, experts and combine in one library call
            return binding.moe_layer_forward(x, w.w_router, w.w13, w.w2, w.k, ws, ws13=w.ws13, ws2=w.ws2,
                                             logits=bufs.get("logits"), topk_idx=bufs.get("idx"), topk_w=bufs.get("w"),
                                             plan=bufs.get("plan"), xp=bufs.get("xp"), h=bufs.get("h"),
                                             y=bufs.get("y"), y_shared=bufs.get("ys"), out=bufs.get("out"),
                                             out_bf16=out_bf16)
        r = binding.moe_route_replay(x, w.w_router, replay_idx, ws, logits=bufs.get("logits"),
                                     topk_w=bufs.get("w"), plan=bufs.get("plan"), xp=bufs.get("xp"))
        f = binding.moe_grouped_ffn(r["xp"], r["plan"], w.w13, w.w2, T, w.k, ws, h=bufs.get("h"), y=bufs.get("y"),
                                    x_shared=x if w.ws13 is not None else None, ws13=w.ws13, ws2=w.ws2,
                                    y_shared=bufs.get("ys"))
        out = binding.moe_combine(f["y"], r["topk_w"], r["plan"], T, w.H, w.E, w.k, y_shared=f["y_shared"],
                                  out=bufs.get("out"), out_bf16=out_bf16)
        return dict(out=out, **r, **f)

    def _run_routed(self, x, ws, bufs, out_bf16, replay_idx):
        """The layer with its experts chosen by w.routing: the same calls with moe_route_topk in three parts."""
        w = self.w
        if replay_idx is not None:
            raise ValueError("router replay needs the softmax top-k router (routing=None)")
        T = x.shape[0]
        logits = binding.moe_router_logits(x, w.w_router, ws, logits=_head(bufs.get("logits"), T))
        plan = bufs.get("plan")
        r = w.routing.select(logits, w.k, ws, _head(bufs.get("idx"), T), _head(bufs.get("w"), T),
                             True if plan is None else plan)
        xp = binding.moe_permute_rows(x, r["plan"], w.E, w.k, xp=_head(bufs.get("xp"), T * w.k))
        f = binding.moe_grouped_ffn(xp, r["plan"], w.w13, w.w2, T, w.k, ws, h=bufs.get("h"), y=bufs.get("y"),
                                    x_shared=x if w.ws13 is not None else None, ws13=w.ws13, ws2=w.ws2,
                                    y_shared=_head(bufs.get("ys"), T))
        out = binding.moe_combine(f["y"], r["topk_w"], r["plan"], T, w.H, w.E, w.k, y_shared=f["y_shared"],
                                  out=_head(bufs.get("out"), T), out_bf16=out_bf16)
        return dict(out=out, logits=logits, xp=xp, **r, **f)

    def _run_fused(self, x, d, out, out_bf16):
        """At most 16 tokens in one kernel; logits and choice into the decode buffers."""
        w, B = self.w, x.shape[0]
        r = w.routing
        chosen = {} if r is None else dict(score=r.score, bias=r.bias, n_group=r.n_group, topk_group=r.topk_group,
                                           renormalize=r.renormalize, scale=r.scale)
        return binding.moe_layer_decode(x, w.w_router, w.w13, w.w2, w.k, d["fused_ws"], w.ws13, w.ws2, out=out,
                                        out_bf16=out_bf16, logits=d["logits"][:B], topk_idx=d["idx"][:B],
                                        topk_w=d["w"][:B], **chosen)["out"]

    def _in_one_kernel(self, x, out_bf16):
        return (self.fused and 0 < x.shape[0] <= binding.DECODE_MAX_TOKENS
                and (out_bf16 is None or not _overlap(x, out_bf16)))

    def _replace(self, ws):
        """A workspace that gives way to a larger one: its status, behind the calls so far on this stream."""
        if ws is not None:
            self._unread.append(ws[:256].clone())

    def check(self):
        """Raise if a kernel of a prefill or decode call since the last check gave up waiting: what it should have written is
        then not there; also of a replay since, of a graph that a caller captured.  Waits for the device.  (DecodeGraphs has a
        check of its own.)"""
        torch.cuda.synchronize(self.w.w13.device)
        spaces = [*self._unread, *self._spaces.values()]
        for d in [self._decode or {}, *self._small.values(), *self._captured]:
            spaces += [d[name] for name in ("ws", "fused_ws") if name in d]
        self._unread = []
        _check_all(spaces)

    def prefill(self, x: torch.Tensor, out_bf16: Optional[torch.Tensor] = None, return_all=False,
                replay_idx: Optional[torch.Tensor] = None):
        """x [T, H] bf16 -> out [T, H] fp32 (optionally also a bf16 copy).  With replay_idx [T, k]
        int32 the recorded expert choices are used instead of the router's own top-k.

        A small batch (at most 1024 tokens) whose intermediates are not returned runs on
        buffers kept for its thread and stream (only `out` is allocated per call): for such
        batches the host's allocations, not the kernels, set the call's latency."""
        T = x.shape[0]
        if not return_all and replay_idx is None and 0 < T <= 1024:
            d = self._small_buffers(T)
            if self._in_one_kernel(x, out_bf16):
                return self._run_fused(x, d, None, out_bf16)
            bufs = {k: d[k] for k in ("logits", "idx", "w", "plan", "xp", "h", "y", "ys")}
            return self._run(x, d["ws"], bufs, out_bf16=out_bf16)["out"]
        res = self._run(x, self._workspace(T), out_bf16=out_bf16, replay_idx=replay_idx)
        return res if return_all else res["out"]

    def backward(self, x: torch.Tensor, fwd: dict, dout: torch.Tensor, weight_grads: bool = True):
        """Backward of the layer for one batch, after ``prefill(x, return_all=True)`` returned ``fwd``.

        dout [T, H] fp32 -> dict(dx [T, H], dw_router, dw13, dw2, dws13, dws2) (fp32), computed by the
        library's combine, grouped-FFN and router backward calls (every reduction in a fixed order,
        no atomics)."""
        w = self.w
        T = x.shape[0]
        ws = self._kept(self._back, binding.backward_workspace_size(T, w.H, w.E, w.k, w.F, w.F_shared))
        c = binding.moe_combine_backward(dout, fwd["y"], fwd["topk_w"], fwd["plan"], w.E, w.k,
                                         dout_bf16=w.ws13 is not None)
        f = binding.moe_grouped_ffn_backward(fwd["xp"], fwd["plan"], w.w13, w.w2, c["dy"], T, w.k, ws,
                                             dw13=weight_grads, dw2=weight_grads,
                                             x_shared=x if w.ws13 is not None else None, ws13=w.ws13, ws2=w.ws2,
                                             dout_bf16=c["dout_bf16"], dws13=weight_grads, dws2=weight_grads)
        if w.routing is None:
            r = binding.moe_route_backward(x, w.w_router, fwd["topk_idx"], fwd["topk_w"], c["dgate"], f["dxp"],
                                           fwd["plan"], ws, dx_shared=f["dx_shared"], dw_router=weight_grads)
        else:
            dlogits = torch.empty_like(fwd["logits"], dtype=torch.bfloat16)
            binding.moe_route_select_backward(fwd["logits"], fwd["topk_idx"], c["dgate"], w.routing.score,
                                              w.routing.renormalize, w.routing.scale, dlogits=False,
                                              dlogits_bf16=dlogits)
            r = binding.moe_router_backward(x, w.w_router, dlogits, f["dxp"], fwd["plan"], w.k, ws,
                                            dx_shared=f["dx_shared"], dw_router=weight_grads)
        binding.check_status(ws)
        return dict(dx=r["dx"], dw_router=r["dw_router"], dw13=f["dw13"], dw2=f["dw2"], dws13=f["dws13"],
                    dws2=f["dws2"], dgate=c["dgate"], dy=c["dy"], dxp=f["dxp"], workspace=ws)

    def alloc_decode(self, max_batch: int):
        """Preallocate decode buffers for up to ``max_batch`` concurrent requests."""
        if _capturing():
            raise RuntimeError("alloc_decode cannot be captured: its workspaces are cleared once, not by every replay")
        for name in ("ws", "fused_ws"):
            self._replace((self._decode or {}).get(name))
        self._decode = self._buffers(max_batch)

    def _decode_buffers(self, B):
        """decode's buffers, of at least B rows.  A captured call keeps those it finds, or is given some of its own: what is
        cleared inside a capture is not clear outside."""
        d, capturing = self._decode, _capturing()
        if d is None or d["B"] < B:
            if capturing:
                d = self._buffers(max(B, 1))
            else:
                self.alloc_decode(max(B, 1))
                d = self._decode
        if capturing and not any(c is d for c in self._captured):
            self._captured.append(d)
        return d

    def _small_buffers(self, T):
        """prefill's buffers of at least T rows: the caller's; a captured call's are its graph's."""
        key = _caller()
        if key is None:
            self._captured.append(self._buffers(T))
            return self._captured[-1]
        d = self._small.get(key)
        if d is None or d["B"] < T:
            for name in ("ws", "fused_ws"):
                self._replace((d or {}).get(name))
            d = self._small[key] = self._buffers(T)
        return d

    def _buffers(self, B):
        w = self.w
        dev = w.w13.device
        S = B * w.k
        d = dict(
            B=B,
            logits=torch.empty((B, w.E), dtype=torch.float32, device=dev),
            idx=torch.empty((B, w.k), dtype=torch.int32, device=dev),
            w=torch.empty((B, w.k), dtype=torch.float32, device=dev),
            plan=torch.empty(binding.plan_len(B, w.E, w.k), dtype=torch.int32, device=dev),
            xp=torch.empty((S, w.H), dtype=torch.bfloat16, device=dev),
            h=torch.empty((S, w.F), dtype=torch.bfloat16, device=dev),
            y=torch.empty((S, w.H), dtype=torch.float32, device=dev),
            ys=torch.empty((B, w.H), dtype=torch.float32, device=dev) if w.ws13 is not None else None,
            out=torch.empty((B, w.H), dtype=torch.float32, device=dev),
            ws=binding.new_workspace(binding.workspace_size(B, w.H, w.E, w.k, w.F, w.F_shared, 0), dev),
        )
        if self.fused:
            few = min(B, binding.DECODE_MAX_TOKENS)
            d["fused_ws"] = binding.new_workspace(
                binding.moe_decode_workspace_size(few, w.H, w.E, w.k, w.F, w.F_shared), dev)
        d["device"] = torch.device(dev)
        p = lambda t: None if t is None else t.data_ptr()   # noqa: E731
        # moe_layer_forward's arguments; decode() fills in x (0), B (6), out_bf16 (21) and the stream (24)
        d["args"] = [None, p(w.w_router), p(w.w13), p(w.w2), p(w.ws13), p(w.ws2), B, w.H, w.E, w.k, w.F, w.F_shared,
                     p(d["logits"]), p(d["idx"]), p(d["w"]), p(d["plan"]), p(d["xp"]), p(d["h"]), p(d["y"]),
                     p(d["ys"]), p(d["out"]), None, p(d["ws"]), d["ws"].numel(), None]
        d["fn"] = binding.lib().moe_layer_forward
        return d

    def decode(self, x_tokens: torch.Tensor, out_bf16: Optional[torch.Tensor] = None) -> torch.Tensor:
        """One token per request: x_tokens [B, H] bf16 -> [B, H] fp32 (a view of the decode buffer);
        out_bf16 [B, H] (optional) receives the bf16 copy the head reads.

        One library call (moe_layer_forward) on buffers allocated once: the argument list is built in
        alloc_decode (every buffer's batch-B view starts at the same address), so a call checks the
        token tensor, sets its pointer, the batch size and the stream, and enters the library."""
        return self._decode_in(self._decode_buffers(x_tokens.shape[0]), x_tokens, out_bf16)

    def _decode_in(self, d, x_tokens, out_bf16=None):
        B, w = x_tokens.shape[0], self.w
        if (x_tokens.dtype != torch.bfloat16 or x_tokens.device != d["device"] or not x_tokens.is_contiguous()
                or x_tokens.dim() != 2 or x_tokens.shape[1] != w.H):
            raise ValueError(f"x_tokens must be a contiguous [B, {w.H}] bf16 tensor on {d['device']}")
        if out_bf16 is not None:
            binding._req(out_bf16, torch.bfloat16, "out_bf16", (B, w.H))
        if self._in_one_kernel(x_tokens, out_bf16):
            return self._run_fused(x_tokens, d, d["out"][:B], out_bf16)
        if w.routing is not None:
            bufs = {name: d[name] for name in ("logits", "idx", "w", "plan", "xp", "h", "y", "ys", "out")}
            return self._run_routed(x_tokens, d["ws"], bufs, out_bf16, None)["out"]
        args = d["args"]
        args[0] = x_tokens.data_ptr()
        args[6] = B
        args[21] = None if out_bf16 is None else out_bf16.data_ptr()
        args[24] = torch.cuda.current_stream(d["device"]).cuda_stream
        binding.check(d["fn"](*args))
        return d["out"][:B]


class InputStager:
    """Double-buffered host-to-device staging of a step's inputs on a side stream.

    ``stage(host)`` issues the copies of the next batch (pinned host tensors) into
    the buffer the step before last has finished with; ``next()`` makes the
    current stream wait for the oldest staged batch and returns its device
    buffers; ``release()`` marks that batch's buffers free once the work enqueued
    so far on the current stream is done.  Staging batch i+1 before running
    batch i overlaps its copies with batch i's kernels.
    """

    def __init__(self, like: dict):
        dev = next(iter(like.values())).device
        self.bufs = [{k: torch.empty_like(v) for k, v in like.items()} for _ in range(2)]
        self.copy_stream = torch.cuda.Stream(device=dev)
        self.ready = [torch.cuda.Event() for _ in range(2)]
        self.free = [torch.cuda.Event() for _ in range(2)]
        self.used = [False, False]
        self.fill = 0
        self.cur = 0

    def stage(self, host: dict):
        b = self.fill
        s = self.copy_stream
        if self.used[b]:
            s.wait_event(self.free[b])
        with torch.cuda.stream(s):
            for k, v in host.items():
                self.bufs[b][k].copy_(v, non_blocking=True)
            self.ready[b].record(s)
        self.fill ^= 1

    def next(self) -> dict:
        b = self.cur
        torch.cuda.current_stream().wait_event(self.ready[b])
        return self.bufs[b]

    def release(self):
        b = self.cur
        self.free[b].record(torch.cuda.current_stream())
        self.used[b] = True
        self.cur ^= 1


class DecodeGraphs:
    """Decode steps captured as CUDA graphs, one per batch-size bucket.

    Every kernel of the decode path takes its sizes and buffers at capture time,
    so a step for a bucket of B requests replays as one graph launch; batches
    smaller than a bucket are padded with zero tokens, which changes no other
    row's bits (every row is computed on its own).  The captured kernels are the
    same as the eager ones, so a replayed step gives the same bits as
    MoELayer.decode on the same tokens.  They read the weights that the layer has
    now and write the buffers it decodes in now: both are kept alive here.
    """

    def __init__(self, layer: MoELayer, buckets=(1, 2, 4, 8, 16, 32, 64, 128)):
        self.layer = layer
        self.buckets = sorted(buckets)
        w = layer.w
        dev = w.w13.device
        layer.alloc_decode(self.buckets[-1])
        # captured kernels hold addresses: a larger batch gives the layer new buffers, these stay the graphs'
        self._bufs = layer._decode
        self._held = [*vars(w).values(), w.routing and w.routing.bias]
        self.inp = {B: torch.zeros((B, w.H), dtype=torch.bfloat16, device=dev) for B in self.buckets}
        self.out = {}
        self.graphs = {}
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for B in self.buckets:
                layer.decode(self.inp[B])          # warm-up outside capture (kernel attributes, caches)
        torch.cuda.current_stream(dev).wait_stream(side)
        for B in self.buckets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.out[B] = layer._decode_in(self._bufs, self.inp[B])
            self.graphs[B] = g

    def __call__(self, x_tokens: torch.Tensor) -> torch.Tensor:
        """x_tokens [b, H] bf16 (b <= largest bucket) -> [b, H] fp32 (a view of the graph's output)."""
        b = x_tokens.shape[0]
        B = next(B for B in self.buckets if B >= b)
        self.inp[B][:b].copy_(x_tokens)
        if b < B:
            self.inp[B][b:].zero_()
        self.graphs[B].replay()
        return self.out[B][:b]

    def check(self):
        """As MoELayer.check, for the replays."""
        torch.cuda.synchronize(self.layer.w.w13.device)
        _check_all([self._bufs[name] for name in ("ws", "fused_ws") if name in self._bufs])


def moe_prefill(layer: MoELayer, x: torch.Tensor) -> torch.Tensor:
    return layer.prefill(x)


def moe_decode(layer: MoELayer, x_tokens: torch.Tensor) -> torch.Tensor:
    return layer.decode(x_tokens)


def head_verify_drafts(hidden, w_vocab, noise, draft_tokens=None, draft_logits=None, accept_u=None, n_draft=None,
                       temperature=1.0, logits=None, workspace=None):
    """The end of a drafted decode step: the head's logits of B requests' D + 1 rows each, then binding.verify_drafts on them.

    hidden [B * (D + 1), H] bf16, request by request, row i of a request the state behind its i-th drafted token (row 0:
    behind its last emitted one); noise [B, V].  Returns verify_drafts' dict and the logits [B, D + 1, V] fp32 (into
    ``logits`` if given).  Without a workspace the dict has the ``workspace`` that the call took: binding.check_status of it,
    as of a given one, raises if the head's kernel gave up waiting, whose logits and tokens are then not to be used."""
    T, H = hidden.shape
    B, V = noise.shape
    D = 0 if draft_tokens is None else draft_tokens.shape[1]
    if T != B * (D + 1) or w_vocab.shape[0] != V:
        raise ValueError(f"hidden must have {B} * {D + 1} rows and w_vocab {V}, got {T} and {w_vocab.shape[0]}")
    need = max(binding.workspace_size(T, H, V=V), binding.verify_workspace_size(B, D, V))
    made = {}
    if workspace is None:
        workspace = made["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=hidden.device)
        workspace[:256].zero_()
    target = torch.zeros(T, dtype=torch.int32, device=hidden.device)     # the head's own logprob is not used
    logits = None if logits is None else logits.view(T, V)
    z = binding.lm_logprob_kl(hidden, w_vocab, target, workspace, logits=logits, write_logits=True)["logits"]
    z = z.view(B, D + 1, V)
    got = binding.verify_drafts(z, noise, workspace, draft_tokens, draft_logits, accept_u, n_draft, temperature)
    return {**got, "logits": z, **made}


def head_logprob_kl(hidden, w_vocab, target, rollout_logp=None, beta=2.0, workspace=None, logits=None,
                    write_logits=False):
    """Token logprobs of the exact target ids, and (with rollout logprobs) k3 and the IcePop mask."""
    T, H = hidden.shape
    V = w_vocab.shape[0]
    if workspace is None:
        workspace = binding.new_workspace(binding.workspace_size(T, H, V=V), hidden.device)
    return binding.lm_logprob_kl(hidden, w_vocab, target, workspace, rollout_logp=rollout_logp, beta=beta,
                                 logits=logits, write_logits=write_logits)
