"""MoE blocks.  The 8-bit one: residual + norm, scored routing, e4m3 experts, combine.

What one block of a transformer does around its MoE layer, with the experts' weights and activations in e4m3 (a scale
per 128 x 128 weights and per row and 128 activations):

    r   = x + residual                          (stored: the residual stream)
    n   = rms_norm(r) * w_norm                  bf16 for the router, e4m3 for the experts, in one pass
    experts and weights from n @ w_router^T     (api.Routing)
    h_e = e4m3(silu(n W_gate) * (n W_up)),  y_e = h_e W_down       for the chosen experts, and for the shared one
    out = sum_j weight_j y_j + y_shared         fp32, fixed order

Every step is per token with one reduction order, so a token's bits do not depend on its batch, on prefill or decode, or
on the kernel that a batch size selects.

MoEBlock is the bf16 block with norms before and after its layer, its gate and residual scale; forward and backward.
"""
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding
from .api import MoELayer, MoEWeights, Routing


@dataclass
class Fp8MoEWeights:
    w_norm: torch.Tensor                    # [H] bf16
    w_router: torch.Tensor                  # [E, H] bf16
    w13: torch.Tensor                       # [E, 2F, H] e4m3 (gate rows, then up rows)
    w13_scale: torch.Tensor                 # [E, 2F/128, ceil(H/128)] fp32
    w2: torch.Tensor                        # [E, H, F] e4m3
    w2_scale: torch.Tensor                  # [E, ceil(H/128), F/128] fp32
    k: int
    routing: Routing
    ws13: Optional[torch.Tensor] = None     # shared expert: [1, 2Fs, H] and [1, H, Fs] e4m3 with their scales
    ws13_scale: Optional[torch.Tensor] = None
    ws2: Optional[torch.Tensor] = None
    ws2_scale: Optional[torch.Tensor] = None
    eps: float = 1e-6

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
        return 0 if self.ws13 is None else self.ws13.shape[1] // 2

    @classmethod
    def from_bf16(cls, w_norm, w_router, w13, w2, k, routing, ws13=None, ws2=None, eps=1e-6):
        """Quantises bf16 expert weights [E, 2F, H], [E, H, F] (shared [2Fs, H], [H, Fs]) once."""
        shared = [None] * 4
        if ws13 is not None:
            shared = [*binding.fp8_quantize(ws13.unsqueeze(0), 128), *binding.fp8_quantize(ws2.unsqueeze(0), 128)]
        return cls(w_norm, w_router, *binding.fp8_quantize(w13, 128), *binding.fp8_quantize(w2, 128), k, routing, *shared,
                   eps=eps)


class Fp8MoEBlock:
    """One 8-bit MoE block on one GPU; see the module's text."""

    def __init__(self, weights: Fp8MoEWeights):
        self.w = weights
        self._bufs = None                       # decode's
        self._ws = {}                           # prefill's workspaces, one per thread and stream
        self._unread, self._captured = [], []   # others with a status that check() reads: replaced ones, graphs'
        self._held = []                         # decode's buffers that a caller's graphs use

    def _workspace(self, T):
        """prefill's workspace: this thread's own on the current stream (calls of two threads interleave their launches), kept
        for its status; a captured call's belongs to its graph."""
        w = self.w
        need = binding.workspace_size(T, w.H, w.E, w.k)
        if torch.cuda.is_current_stream_capturing():
            self._captured.append(binding.new_workspace(need, w.w13.device))
            return self._captured[-1]
        key = threading.get_ident(), binding._stream()
        ws = self._ws.get(key)
        if ws is None or ws.numel() < need:
            if ws is not None:
                self._unread.append(ws)
            ws = self._ws[key] = binding.new_workspace(need, w.w13.device)
        return ws

    def _alloc(self, T, kept):
        """The intermediates of a batch of T tokens."""
        w, dev = self.w, self.w.w13.device
        S, nb = T * w.k, (w.H + 127) // 128
        e = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)   # noqa: E731
        b = dict(T=T, norm=e((T, w.H), torch.bfloat16), q=e((T, w.H), binding.FP8), q_scale=e((T, nb)), rstd=e((T,)),
                 logits=e((T, w.E)), topk_idx=e((T, w.k), torch.int32), topk_w=e((T, w.k)),
                 plan=e(binding.plan_len(T, w.E, w.k), torch.int32), xp=e((S, w.H), binding.FP8), xp_scale=e((S, nb)),
                 h=e((S, w.F), binding.FP8), h_scale=e((S, w.F // 128)), y=e((S, w.H)),
                 residual=None, out=None)
        if w.F_shared:
            b.update(hs=e((T, w.F_shared), binding.FP8), hs_scale=e((T, w.F_shared // 128)), ys=e((T, w.H)))
        if kept:
            b.update(residual=e((T, w.H), torch.bfloat16), out=e((T, w.H)),
                     ws=binding.new_workspace(binding.workspace_size(T, w.H, w.E, w.k), dev))
        else:
            b["ws"] = self._workspace(T)
        return b

    def _run(self, x, residual, b, residual_out, out, out_bf16):
        w = self.w
        T = x.shape[0]
        S = T * w.k
        ws = b["ws"]
        n = binding.add_rms_norm(x, w.w_norm, residual, w.eps, out=b["norm"][:T], fp8=True, residual_out=residual_out,
                                 q=b["q"][:T], scale=b["q_scale"][:T], rstd=b["rstd"][:T])
        logits = binding.moe_router_logits(n["out"], w.w_router, ws, logits=b["logits"][:T])
        r = w.routing.select(logits, w.k, ws, b["topk_idx"][:T], b["topk_w"][:T], b["plan"])
        xp, xs = binding.moe_permute_fp8(n["q"], n["scale"], r["plan"], w.E, w.k, b["xp"][:S], b["xp_scale"][:S])
        h = binding.moe_grouped_swiglu_fp8(xp, xs, r["plan"], w.w13, w.w13_scale, T, w.k, ws, b["h"][:S], b["h_scale"][:S])
        y = binding.moe_grouped_down_fp8(h["h"], h["h_scale"], r["plan"], w.w2, w.w2_scale, T, w.k, ws, b["y"][:S])
        ys = None
        if w.F_shared:
            hs = binding.moe_grouped_swiglu_fp8(n["q"], n["scale"], None, w.ws13, w.ws13_scale, T, 1, ws, b["hs"][:T],
                                                b["hs_scale"][:T])
            ys = binding.moe_grouped_down_fp8(hs["h"], hs["h_scale"], None, w.ws2, w.ws2_scale, T, 1, ws, b["ys"][:T])
        out = binding.moe_combine(y, r["topk_w"], r["plan"], T, w.H, w.E, w.k, y_shared=ys, out=out, out_bf16=out_bf16)
        return dict(out=out, residual=n["residual"] if residual is not None else x, norm=n["out"], q=n["q"],
                    q_scale=n["scale"], rstd=n["rstd"], logits=logits, topk_idx=r["topk_idx"], topk_w=r["topk_w"],
                    plan=r["plan"], xp=xp, xp_scale=xs, h=h["h"], h_scale=h["h_scale"], y=y, y_shared=ys, workspace=ws)

    def prefill(self, x, residual=None, residual_out=None, out_bf16=None, return_all=False):
        """x [T, H] (bf16 or fp32) and residual [T, H] -> (out [T, H] fp32, the new residual [T, H]).

        residual_out may be residual itself; without a residual x is the residual stream.  return_all: the dict of every
        intermediate instead."""
        T = x.shape[0]
        res = self._run(x, residual, self._alloc(T, False), residual_out, None, out_bf16)
        return res if return_all else (res["out"], res["residual"])

    def decode(self, x, residual, out_bf16=None):
        """One token per request: as prefill, for a bf16 residual, on buffers kept for the largest batch so far.

        Returns views of those buffers: (out [B, H] fp32, residual [B, H] bf16), valid until the next call, which may be
        given them or rows of them.  The calls share the buffers, so they belong on one stream.  Those that a captured call
        uses live as long as the block."""
        B, b, capturing = x.shape[0], self._bufs, torch.cuda.is_current_stream_capturing()
        if b is None or b["T"] < B:
            new = self._alloc(max(B, 1), True)
            if not capturing:                   # (what is cleared inside a capture is not clear outside)
                if b is not None:
                    self._unread.append(b["ws"])
                self._bufs = new
            b = new
        if capturing and not any(h is b for h in self._held):
            self._held.append(b)
        # rows of the last step's residual at other places than they go to: a block would write what another one reads
        if (residual is not None and residual.data_ptr() != b["residual"].data_ptr()
                and residual.untyped_storage().data_ptr() == b["residual"].untyped_storage().data_ptr()):
            residual = residual.clone()
        res = self._run(x, residual, b, b["residual"][:B], b["out"][:B], out_bf16)
        return res["out"], res["residual"]

    def check(self):
        """Raise if a kernel of a prefill or decode call since the last check gave up waiting: what it should have written
        is then not there.  Waits for the device."""
        torch.cuda.synchronize(self.w.w13.device)
        spaces = [*self._ws.values(), *self._unread, *self._captured, *(b["ws"] for b in self._held)]
        if self._bufs is not None:
            spaces.append(self._bufs["ws"])
        self._unread = []
        failed = None
        for ws in spaces:                       # all of them, so that each time-out is reported once
            try:
                binding.check_status(ws)
            except RuntimeError as e:
                failed = e
        if failed is not None:
            raise failed


class Fp8DecodeGraph:
    """A decode step of B requests as one CUDA graph: fill x and residual, replay, read out and residual_out.

    The captured kernels are those of Fp8MoEBlock.decode, so the bits are the same.  They read the weights that the block
    has now: a graph keeps those alive, and is made anew for others."""

    def __init__(self, block: Fp8MoEBlock, B: int, x_dtype=torch.bfloat16):
        w, dev = block.w, block.w.w13.device
        # captured kernels hold addresses: the tensors live as long as the graph, whatever becomes of block and weights
        self._held = [*vars(w).values(), w.routing.bias]
        self.x = torch.zeros((B, w.H), dtype=x_dtype, device=dev)
        self.residual = torch.zeros((B, w.H), dtype=torch.bfloat16, device=dev)
        bufs = block._alloc(B, True)
        run = lambda: block._run(self.x, self.residual, bufs, bufs["residual"], bufs["out"], None)   # noqa: E731
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            run()                               # warm-up outside the capture (kernel attributes, caches)
        torch.cuda.current_stream(dev).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            run()
        self._bufs = bufs
        self.out, self.residual_out = bufs["out"], bufs["residual"]

    def replay(self):
        self.graph.replay()
        return self.out, self.residual_out

    def check(self):
        """As Fp8MoEBlock.check, for the replays."""
        torch.cuda.synchronize(self.x.device)
        binding.check_status(self._bufs["ws"])


@dataclass
class MoEBlockWeights:
    layer: MoEWeights
    w_post: torch.Tensor                    # [H] bf16: the norm of the layer's output
    w_next: Optional[torch.Tensor] = None   # [H] bf16: the next block's norm; None behind the last block
    gate: Optional[torch.Tensor] = None     # [H] bf16, a channel's
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    eps: float = 1e-6


class MoEBlock:
    """One bf16 MoE block with norms before and after its layer, from one normalised row to the next block's:

        m   = MoE layer of n                                               (api.MoELayer)
        r'  = residual_scale r + branch_scale gate rms_norm(m) w_post      the residual stream
        n'  = rms_norm(r') w_next                                          bf16, the next block's n

    The norms, gate and scales are one call (binding.sandwich_norm).  The first block's n is add_rms_norm's of the embedded
    row.  Every step is per token with one reduction order, so prefill and decode give the same bits.

    prefill and backward may run on several threads and streams at once.  A graph that a caller captures needs the block and
    its weights kept, as MoELayer's."""

    def __init__(self, weights: MoEBlockWeights, fused: Optional[bool] = None):
        """fused: decode of at most 16 rows runs the layer in one kernel (MoELayer); None: where its weights fit."""
        self.w = weights
        self.layer = MoELayer(weights.layer, fused=fused)

    def _after(self, m, residual, gate, residual_out=None):
        w = self.w
        return binding.sandwich_norm(m, w.w_post, residual, w.w_next, w.gate if gate is None else gate, w.residual_scale,
                                     w.branch_scale, w.eps, residual_out=residual_out)

    def prefill(self, n, residual, gate=None, residual_out=None, return_all=False):
        """n [T, H] bf16 and residual [T, H] (bf16 or fp32) -> (n' or None, the new residual).

        gate [T] fp32: one per token, in the place of the weights'.  return_all: the dict that backward takes."""
        m = self.layer.prefill(n, return_all=return_all)
        s = self._after(m["out"] if return_all else m, residual, gate, residual_out)
        if return_all:
            return {**s, "layer": m, "n": n, "gate": self.w.gate if gate is None else gate}
        return s["out"], s["residual"]

    def decode(self, n, residual, gate=None, residual_out=None):
        """One row per request (or per drafted token): as prefill, the layer on buffers kept for the largest batch so far.
        The calls share those buffers, so they belong on one stream."""
        s = self._after(self.layer.decode(n), residual, gate, residual_out)
        return s["out"], s["residual"]

    def backward(self, fwd, dnext, dres=None, weight_grads=True):
        """fwd: prefill(..., return_all=True)'s dict; dnext [T, H]: the gradient of n' (None behind the last block); dres: the
        gradient that reaches the new residual from the stream, in its type.

        Returns the gradients dn (of n, fp32), dresidual, dw_post, dw_next, dgate and the layer's (``layer``)."""
        w = self.w
        # a call's own: between its two kernels nobody else's partial sums may get there
        ws = torch.empty(binding.sandwich_norm_backward_workspace_size(*fwd["residual"].shape), dtype=torch.uint8,
                         device=fwd["residual"].device)
        ws[:256].zero_()
        s = binding.sandwich_norm_backward(dnext, dres, fwd["layer"]["out"], w.w_post, fwd["rstd_post"], fwd["residual"],
                                           w.w_next if dnext is not None else None, fwd["rstd"] if dnext is not None else None,
                                           fwd["gate"], w.residual_scale, w.branch_scale, dweights=weight_grads,
                                           workspace=ws)
        g = self.layer.backward(fwd["n"], fwd["layer"], s["dx"], weight_grads)     # (waits for the GPU)
        binding.check_status(ws)
        return dict(dn=g["dx"], dresidual=s["dresidual"], dw_post=s["dw_post"], dw_next=s["dw_next"], dgate=s["dgate"], layer=g)

    def check(self):
        """MoELayer.check."""
        self.layer.check()
