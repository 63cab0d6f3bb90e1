"""Python binding of the C ABI: argument marshalling only.

Each function checks dtypes/devices/contiguity, allocates missing outputs with
torch (device memory only), passes raw pointers and the current CUDA stream to
libinvmoe.so and raises on a non-zero status.  No arithmetic of the hot path
happens here: every step runs in the library's kernels.
"""
import ctypes
import math

import torch

from ._lib import check, lib, marshal


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    # the raw handle: building a torch.cuda.Stream object costs 2.9 us of a call's 8-20 us on the host, this 0.4
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _req(t, dtype, name, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    # the library launches on the current device: a pointer into another GPU's memory
    # must not reach a kernel
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current CUDA device is cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _opt(t, dtype, name, shape=None):
    """_req for an optional tensor (None passes)."""
    return None if t is None else _req(t, dtype, name, shape)


def _req_plan(plan, T, E, k):
    _req(plan, torch.int32, "plan")
    if plan.numel() < plan_len(T, E, k):
        raise ValueError("plan is too small")
    return plan


def plan_len(T, E, k) -> int:
    return int(lib().invmoe_plan_len(T, E, k))


def workspace_size(T, H, E=0, k=0, F=0, F_shared=0, V=0) -> int:
    return int(lib().invmoe_workspace_size(T, H, E, k, F, F_shared, V))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled device workspace (the first 256 bytes are the status word)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def check_status(workspace: torch.Tensor):
    """Synchronise the current stream and raise if a kernel's bounded wait ran out."""
    check(lib().invmoe_check(_p(workspace), _stream()))


def moe_route_topk(x, w_router, k, workspace, logits=None, topk_idx=None, topk_w=None, plan=None, xp=None):
    T, H = x.shape
    E = w_router.shape[0]
    dev = x.device
    _req(x, torch.bfloat16, "x")
    _req(w_router, torch.bfloat16, "w_router", (E, H))
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if logits is None else logits
    topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev) if topk_idx is None else topk_idx
    topk_w = torch.empty((T, k), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    plan = torch.empty(plan_len(T, E, k), dtype=torch.int32, device=dev) if plan is None else plan
    xp = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev) if xp is None else xp
    _req(logits, torch.float32, "logits", (T, E))
    _req(topk_idx, torch.int32, "topk_idx", (T, k))
    _req(topk_w, torch.float32, "topk_w", (T, k))
    _req(plan, torch.int32, "plan")
    if plan.numel() < plan_len(T, E, k):
        raise ValueError("plan is too small")
    _req(xp, torch.bfloat16, "xp")
    if xp.numel() < T * k * H:
        raise ValueError("xp is too small")
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_route_topk(_p(x), _p(w_router), T, H, E, k, _p(logits), _p(topk_idx), _p(topk_w), _p(plan),
                               _p(xp), _p(workspace), workspace.numel(), _stream()))
    return dict(logits=logits, topk_idx=topk_idx, topk_w=topk_w, plan=plan, xp=xp)


def moe_route_replay(x, w_router, topk_idx, workspace, logits=None, topk_w=None, plan=None, xp=None):
    """Router replay: the given experts [T, k] int32, fresh gates, plan and permuted rows."""
    T, H = x.shape
    E = w_router.shape[0]
    k = topk_idx.shape[1]
    dev = x.device
    _req(x, torch.bfloat16, "x")
    _req(w_router, torch.bfloat16, "w_router", (E, H))
    _req(topk_idx, torch.int32, "topk_idx", (T, k))
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if logits is None else logits
    topk_w = torch.empty((T, k), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    plan = torch.empty(plan_len(T, E, k), dtype=torch.int32, device=dev) if plan is None else plan
    xp = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev) if xp is None else xp
    _req(logits, torch.float32, "logits", (T, E))
    _req(topk_w, torch.float32, "topk_w", (T, k))
    _req(plan, torch.int32, "plan")
    _req(xp, torch.bfloat16, "xp")
    if plan.numel() < plan_len(T, E, k) or xp.numel() < T * k * H:
        raise ValueError("plan / xp too small")
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_route_replay(_p(x), _p(w_router), _p(topk_idx), T, H, E, k, _p(logits), _p(topk_w), _p(plan),
                                 _p(xp), _p(workspace), workspace.numel(), _stream()))
    return dict(logits=logits, topk_idx=topk_idx, topk_w=topk_w, plan=plan, xp=xp)


def moe_grouped_ffn(xp, plan, w13, w2, T, k, workspace, h=None, y=None,
                    x_shared=None, ws13=None, ws2=None, y_shared=None):
    E, F2, H = w13.shape
    F = F2 // 2
    dev = xp.device
    S = T * k
    _req(xp, torch.bfloat16, "xp")
    _req(plan, torch.int32, "plan")
    _req(w13, torch.bfloat16, "w13")
    _req(w2, torch.bfloat16, "w2", (E, H, F))
    h = torch.empty((S, F), dtype=torch.bfloat16, device=dev) if h is None else h
    y = torch.empty((S, H), dtype=torch.float32, device=dev) if y is None else y
    _req(h, torch.bfloat16, "h")
    _req(y, torch.float32, "y")
    if h.numel() < S * F or y.numel() < S * H:
        raise ValueError("h / y too small")
    Fs = 0
    if ws13 is not None:
        Fs = ws13.shape[0] // 2
        _req(x_shared, torch.bfloat16, "x_shared", (T, H))
        _req(ws13, torch.bfloat16, "ws13", (2 * Fs, H))
        _req(ws2, torch.bfloat16, "ws2", (H, Fs))
        y_shared = torch.empty((T, H), dtype=torch.float32, device=dev) if y_shared is None else y_shared
        _req(y_shared, torch.float32, "y_shared", (T, H))
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_grouped_ffn(_p(xp), _p(plan), _p(w13), _p(w2), T, H, E, k, F, _p(h), _p(y),
                                _p(x_shared), _p(ws13), _p(ws2), Fs, _p(y_shared), _p(workspace),
                                workspace.numel(), _stream()))
    return dict(h=h, y=y, y_shared=y_shared)


def moe_layer_forward(x, w_router, w13, w2, k, workspace, ws13=None, ws2=None, logits=None, topk_idx=None, topk_w=None,
                      plan=None, xp=None, h=None, y=None, y_shared=None, out=None, out_bf16=None):
    """The whole layer in one library call (route, grouped SwiGLU experts, combine); missing outputs
    are allocated.  Returns the same dict as the three calls."""
    T, H = x.shape
    E, F2, _ = w13.shape
    F = F2 // 2
    Fs = 0 if ws13 is None else ws13.shape[0] // 2
    S = T * k
    dev = x.device
    _req(x, torch.bfloat16, "x")
    _req(w_router, torch.bfloat16, "w_router", (E, H))
    _req(w13, torch.bfloat16, "w13", (E, 2 * F, H))
    _req(w2, torch.bfloat16, "w2", (E, H, F))

    def buf(t, shape, dtype, name, min_numel=None):
        t = torch.empty(shape, dtype=dtype, device=dev) if t is None else t
        _req(t, dtype, name)
        if t.numel() < (min_numel if min_numel is not None else math.prod(shape)):
            raise ValueError(f"{name} is too small")
        return t
    logits = buf(logits, (T, E), torch.float32, "logits")
    topk_idx = buf(topk_idx, (T, k), torch.int32, "topk_idx")
    topk_w = buf(topk_w, (T, k), torch.float32, "topk_w")
    plan = buf(plan, (plan_len(T, E, k),), torch.int32, "plan")
    xp = buf(xp, (S, H), torch.bfloat16, "xp")
    h = buf(h, (S, F), torch.bfloat16, "h")
    y = buf(y, (S, H), torch.float32, "y")
    out = buf(out, (T, H), torch.float32, "out")
    if Fs:
        _req(ws13, torch.bfloat16, "ws13", (2 * Fs, H))
        _req(ws2, torch.bfloat16, "ws2", (H, Fs))
        y_shared = buf(y_shared, (T, H), torch.float32, "y_shared")
    else:
        y_shared = None
    _opt(out_bf16, torch.bfloat16, "out_bf16", (T, H))
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_layer_forward(_p(x), _p(w_router), _p(w13), _p(w2), _p(ws13), _p(ws2), T, H, E, k, F, Fs,
                                  _p(logits), _p(topk_idx), _p(topk_w), _p(plan), _p(xp), _p(h), _p(y), _p(y_shared),
                                  _p(out), _p(out_bf16), _p(workspace), workspace.numel(), _stream()))
    return dict(out=out, logits=logits, topk_idx=topk_idx, topk_w=topk_w, plan=plan, xp=xp, h=h, y=y,
                y_shared=y_shared)


def moe_combine(y, topk_w, plan, T, H, E, k, y_shared=None, out=None, out_bf16=None):
    dev = y.device
    _req(y, torch.float32, "y")
    _req(topk_w, torch.float32, "topk_w", (T, k))
    _req(plan, torch.int32, "plan")
    if y_shared is not None:
        _req(y_shared, torch.float32, "y_shared", (T, H))
    out = torch.empty((T, H), dtype=torch.float32, device=dev) if out is None else out
    _req(out, torch.float32, "out", (T, H))
    if out_bf16 is not None:
        _req(out_bf16, torch.bfloat16, "out_bf16", (T, H))
    check(lib().moe_combine(_p(y), _p(topk_w), _p(plan), _p(y_shared), T, H, E, k, _p(out), _p(out_bf16),
                            _stream()))
    return out


def lm_logprob_kl(hidden, w_vocab, target, workspace, rollout_logp=None, beta=2.0, logits=None,
                  logp=None, lse=None, k3=None, mask=None, write_logits=False):
    """logits are written only if a buffer is passed or write_logits is set."""
    T, H = hidden.shape
    V = w_vocab.shape[0]
    dev = hidden.device
    _req(hidden, torch.bfloat16, "hidden")
    _req(w_vocab, torch.bfloat16, "w_vocab", (V, H))
    _req(target, torch.int32, "target", (T,))
    if logits is None and write_logits:
        logits = torch.empty((T, V), dtype=torch.float32, device=dev)
    if logits is not None:
        _req(logits, torch.float32, "logits", (T, V))
    logp = torch.empty(T, dtype=torch.float32, device=dev) if logp is None else logp
    lse = torch.empty(T, dtype=torch.float32, device=dev) if lse is None else lse
    if rollout_logp is not None:
        _req(rollout_logp, torch.float32, "rollout_logp", (T,))
        k3 = torch.empty(T, dtype=torch.float32, device=dev) if k3 is None else k3
        mask = torch.empty(T, dtype=torch.uint8, device=dev) if mask is None else mask
        _req(k3, torch.float32, "k3", (T,))
        _req(mask, torch.uint8, "mask", (T,))
    _req(logp, torch.float32, "logp", (T,))
    _req(lse, torch.float32, "lse", (T,))
    _req(workspace, torch.uint8, "workspace")
    check(lib().lm_logprob_kl(_p(hidden), _p(w_vocab), _p(target), _p(rollout_logp), T, H, V, float(beta),
                              _p(logits), _p(logp), _p(lse), _p(k3), _p(mask), _p(workspace), workspace.numel(),
                              _stream()))
    return dict(logits=logits, logp=logp, lse=lse, k3=k3, mask=mask)


def lm_logprob_partials(hidden, w_vocab_shard, target, V, v0, workspace, partials, tgt_logit, logits=None):
    """Pass 1 of the log-sum-exp on the vocabulary shard [v0, v0 + rows of w_vocab_shard).

    partials: fp32 [T, P, 2] (P >= the shard's chunk count), the shard's chunk j of token t at
    partials[t, j]; tgt_logit [T] fp32 receives z[t, target[t]] where the target is in the shard;
    logits (optional) is the whole [T, V] fp32 array, of which the shard's columns are written."""
    T, H = hidden.shape
    v1 = v0 + w_vocab_shard.shape[0]
    _req(hidden, torch.bfloat16, "hidden")
    _req(w_vocab_shard, torch.bfloat16, "w_vocab_shard", (v1 - v0, H))
    _req(target, torch.int32, "target", (T,))
    _req(partials, torch.float32, "partials")
    if partials.dim() != 3 or partials.shape[0] != T or partials.shape[2] != 2:
        raise ValueError(f"partials must be [T, P, 2], got {tuple(partials.shape)}")
    _req(tgt_logit, torch.float32, "tgt_logit", (T,))
    _opt(logits, torch.float32, "logits", (T, V))
    _req(workspace, torch.uint8, "workspace")
    check(lib().lm_logprob_partials(_p(hidden), _p(w_vocab_shard), _p(target), T, H, V, v0, v1, _p(logits),
                                    _p(partials), partials.shape[1], _p(tgt_logit), _p(workspace), workspace.numel(),
                                    _stream()))
    return partials


def lm_logprob_merge(partials, tgt_logit, target, V, rollout_logp=None, beta=2.0):
    """Pass 2 and the per-token outputs from partials [T, NCH, 2] with target logits [T] (one array),
    or from partials [n, T, P, 2] with target logits [n, T] (n gathered shards of P chunks each)."""
    _req(partials, torch.float32, "partials")
    if partials.dim() == 3:
        T, P = partials.shape[0], partials.shape[1]
        stride, tstride = 0, 0
        _req(tgt_logit, torch.float32, "tgt_logit", (T,))
    elif partials.dim() == 4:
        n, T, P = partials.shape[0], partials.shape[1], partials.shape[2]
        stride, tstride = T * P, T
        _req(tgt_logit, torch.float32, "tgt_logit", (n, T))
    else:
        raise ValueError("partials must be [T, NCH, 2] or [n, T, P, 2]")
    if partials.shape[-1] != 2:
        raise ValueError("partials must end in a (max, sum) pair")
    dev = partials.device
    _req(target, torch.int32, "target", (T,))
    out = dict(logp=torch.empty(T, dtype=torch.float32, device=dev),
               lse=torch.empty(T, dtype=torch.float32, device=dev), k3=None, mask=None)
    if rollout_logp is not None:
        _req(rollout_logp, torch.float32, "rollout_logp", (T,))
        out["k3"] = torch.empty(T, dtype=torch.float32, device=dev)
        out["mask"] = torch.empty(T, dtype=torch.uint8, device=dev)
    check(lib().lm_logprob_merge(_p(partials), P, P, stride, _p(tgt_logit), tstride, _p(target), _p(rollout_logp), T,
                                 V, float(beta), _p(out["logp"]), _p(out["lse"]), _p(out["k3"]), _p(out["mask"]),
                                 _stream()))
    return out


def moe_ep_regroup(recv_xp, recv_counts, workspace, xp_local=None, plan_local=None, row_src=None):
    """Received rows (source-major) -> expert-major rows, the local plan and the row map.

    recv_xp [R, H] bf16, recv_counts [n_src, E_local] int32 (device)."""
    R, H = recv_xp.shape
    n_src, E_local = recv_counts.shape
    dev = recv_xp.device
    _req(recv_xp, torch.bfloat16, "recv_xp")
    _req(recv_counts, torch.int32, "recv_counts")
    xp_local = torch.empty((R, H), dtype=torch.bfloat16, device=dev) if xp_local is None else xp_local
    plan_local = torch.empty(2 * E_local + 1, dtype=torch.int32, device=dev) if plan_local is None else plan_local
    row_src = torch.empty(max(R, 1), dtype=torch.int32, device=dev) if row_src is None else row_src
    _req(xp_local, torch.bfloat16, "xp_local", (R, H))
    _req(plan_local, torch.int32, "plan_local", (2 * E_local + 1,))
    _req(row_src, torch.int32, "row_src")
    if row_src.numel() < R:
        raise ValueError("row_src is too small")
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_ep_regroup(_p(recv_xp), _p(recv_counts), n_src, E_local, R, H, _p(xp_local), _p(plan_local),
                               _p(row_src), _p(workspace), workspace.numel(), _stream()))
    return dict(xp_local=xp_local, plan_local=plan_local, row_src=row_src)


def moe_ep_ungroup(y_local, row_src, y_send=None):
    """y_send[row_src[i]] = y_local[i]: expert outputs back in the received order."""
    R, H = y_local.shape
    _req(y_local, torch.float32, "y_local")
    _req(row_src, torch.int32, "row_src")
    y_send = torch.empty_like(y_local) if y_send is None else y_send
    _req(y_send, torch.float32, "y_send", (R, H))
    check(lib().moe_ep_ungroup(_p(y_local), _p(row_src), R, H, _p(y_send), _stream()))
    return y_send


def moe_shared_expert(x, ws13, ws2, workspace, y_shared=None):
    """The shared expert alone: y_shared [T, H] fp32 = SwiGLU(x)."""
    T, H = x.shape
    Fs = ws13.shape[0] // 2
    _req(x, torch.bfloat16, "x")
    _req(ws13, torch.bfloat16, "ws13", (2 * Fs, H))
    _req(ws2, torch.bfloat16, "ws2", (H, Fs))
    y_shared = torch.empty((T, H), dtype=torch.float32, device=x.device) if y_shared is None else y_shared
    _req(y_shared, torch.float32, "y_shared", (T, H))
    _req(workspace, torch.uint8, "workspace")
    check(lib().moe_shared_expert(_p(x), _p(ws13), _p(ws2), T, H, Fs, _p(y_shared), _p(workspace), workspace.numel(),
                                  _stream()))
    return y_shared


def rl_token_loss(logp_train, logp_rollout, advantage, logp_old=None, beta=2.0, eps_low=0.2, eps_high=0.28):
    """IcePop-masked clipped policy loss per token (+ fixed-order mean), IcePop mask, DIS weights."""
    T = logp_train.shape[0]
    dev = logp_train.device
    for name, t in (("logp_train", logp_train), ("logp_rollout", logp_rollout), ("advantage", advantage)):
        _req(t, torch.float32, name, (T,))
    if logp_old is not None:
        _req(logp_old, torch.float32, "logp_old", (T,))
    out = dict(loss=torch.empty(T, dtype=torch.float32, device=dev),
               loss_mean=torch.empty(1, dtype=torch.float32, device=dev),
               icepop_mask=torch.empty(T, dtype=torch.uint8, device=dev),
               dis_weight=torch.empty(T, dtype=torch.float32, device=dev),
               grad_logp=torch.empty(T, dtype=torch.float32, device=dev))
    check(lib().rl_token_loss(_p(logp_train), _p(logp_old), _p(logp_rollout), _p(advantage), T, float(beta),
                              float(eps_low), float(eps_high), _p(out["icepop_mask"]), _p(out["dis_weight"]),
                              _p(out["loss"]), _p(out["loss_mean"]), _p(out["grad_logp"]), _stream()))
    return out


def lm_head_backward(hidden, w_vocab, target, lse, grad_logp, workspace, dlogits=None, d_hidden=True,
                     d_wvocab=True):
    """Head backward: dlogits [T, V] bf16, d_hidden [T, H] fp32, d_wvocab [V, H] fp32.

    d_hidden / d_wvocab: a tensor to write into, True to allocate one, False to skip it."""
    T, H = hidden.shape
    V = w_vocab.shape[0]
    dev = hidden.device
    _req(hidden, torch.bfloat16, "hidden")
    _req(w_vocab, torch.bfloat16, "w_vocab", (V, H))
    _req(target, torch.int32, "target", (T,))
    _req(lse, torch.float32, "lse", (T,))
    _req(grad_logp, torch.float32, "grad_logp", (T,))
    _req(workspace, torch.uint8, "workspace")
    dlogits = torch.empty((T, V), dtype=torch.bfloat16, device=dev) if dlogits is None else dlogits
    _req(dlogits, torch.bfloat16, "dlogits", (T, V))
    if d_hidden is True:
        d_hidden = torch.empty((T, H), dtype=torch.float32, device=dev)
    if d_wvocab is True:
        d_wvocab = torch.empty((V, H), dtype=torch.float32, device=dev)
    d_hidden = None if d_hidden is False else d_hidden
    d_wvocab = None if d_wvocab is False else d_wvocab
    if d_hidden is not None:
        _req(d_hidden, torch.float32, "d_hidden", (T, H))
    if d_wvocab is not None:
        _req(d_wvocab, torch.float32, "d_wvocab", (V, H))
    check(lib().lm_head_backward(_p(hidden), _p(w_vocab), _p(target), _p(lse), _p(grad_logp), T, H, V,
                                 _p(dlogits), _p(d_hidden), _p(d_wvocab), _p(workspace), workspace.numel(),
                                 _stream()))
    return dict(dlogits=dlogits, d_hidden=d_hidden, d_wvocab=d_wvocab)


def backward_workspace_size(T, H, E, k, F, F_shared=0) -> int:
    return int(lib().invmoe_backward_workspace_size(T, H, E, k, F, F_shared))


def moe_combine_backward(dout, y, topk_w, plan, E, k, dy=None, dgate=None, dout_bf16=False):
    """dy [T*k, H] bf16 (permuted rows), dgate [T, k] fp32, optionally dout_bf16 [T, H] bf16."""
    T, H = dout.shape
    dev = dout.device
    _req(dout, torch.float32, "dout")
    _req(y, torch.float32, "y", (T * k, H))
    _req(topk_w, torch.float32, "topk_w", (T, k))
    _req_plan(plan, T, E, k)
    dy = torch.empty((T * k, H), dtype=torch.bfloat16, device=dev) if dy is None else dy
    dgate = torch.empty((T, k), dtype=torch.float32, device=dev) if dgate is None else dgate
    db = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if dout_bf16 is True else (dout_bf16 or None)
    _req(dy, torch.bfloat16, "dy", (T * k, H))
    _req(dgate, torch.float32, "dgate", (T, k))
    _opt(db, torch.bfloat16, "dout_bf16", (T, H))
    check(lib().moe_combine_backward(_p(dout), _p(y), _p(topk_w), _p(plan), T, H, E, k, _p(dy), _p(dgate), _p(db),
                                     _stream()))
    return dict(dy=dy, dgate=dgate, dout_bf16=db)


def moe_grouped_ffn_backward(xp, plan, w13, w2, dy, T, k, workspace, dxp=None, dw13=True, dw2=True,
                             x_shared=None, ws13=None, ws2=None, dout_bf16=None, dx_shared=None, dws13=True,
                             dws2=True):
    """dxp [T*k, H] fp32, dw13 [E, 2F, H], dw2 [E, H, F] (+ shared: dx_shared, dws13, dws2), all fp32.
    A weight-gradient argument may be a tensor, True (allocate) or False (skip)."""
    E, F2, H = w13.shape
    F = F2 // 2
    dev = xp.device
    S = T * k
    Fs = 0 if ws13 is None else ws13.shape[0] // 2
    _req(xp, torch.bfloat16, "xp", (S, H))
    _req(w13, torch.bfloat16, "w13")
    _req(w2, torch.bfloat16, "w2", (E, H, F))
    _req(dy, torch.bfloat16, "dy", (S, H))
    _req_plan(plan, T, E, k)
    _req(workspace, torch.uint8, "workspace")

    def alloc(v, shape):
        if v is True:
            return torch.empty(shape, dtype=torch.float32, device=dev)
        return None if v is False or v is None else v

    dxp = torch.empty((S, H), dtype=torch.float32, device=dev) if dxp is None else dxp
    dw13, dw2 = alloc(dw13, (E, 2 * F, H)), alloc(dw2, (E, H, F))
    _req(dxp, torch.float32, "dxp", (S, H))
    _opt(dw13, torch.float32, "dw13", (E, 2 * F, H))
    _opt(dw2, torch.float32, "dw2", (E, H, F))
    if Fs:
        _req(x_shared, torch.bfloat16, "x_shared", (T, H))
        _req(ws13, torch.bfloat16, "ws13", (2 * Fs, H))
        _req(ws2, torch.bfloat16, "ws2", (H, Fs))
        _req(dout_bf16, torch.bfloat16, "dout_bf16", (T, H))
        dx_shared = torch.empty((T, H), dtype=torch.float32, device=dev) if dx_shared is None else dx_shared
        dws13, dws2 = alloc(dws13, (2 * Fs, H)), alloc(dws2, (H, Fs))
        _req(dx_shared, torch.float32, "dx_shared", (T, H))
        _opt(dws13, torch.float32, "dws13", (2 * Fs, H))
        _opt(dws2, torch.float32, "dws2", (H, Fs))
    else:
        dx_shared = dws13 = dws2 = None
    check(lib().moe_grouped_ffn_backward(_p(xp), _p(plan), _p(w13), _p(w2), _p(dy), T, H, E, k, F, _p(dxp), _p(dw13),
                                         _p(dw2), _p(x_shared), _p(ws13), _p(ws2), _p(dout_bf16), Fs, _p(dx_shared),
                                         _p(dws13), _p(dws2), _p(workspace), workspace.numel(), _stream()))
    return dict(dxp=dxp, dw13=dw13, dw2=dw2, dx_shared=dx_shared, dws13=dws13, dws2=dws2)


def moe_route_backward(x, w_router, topk_idx, topk_w, dgate, dxp, plan, workspace, dx_shared=None, dx=None,
                       dw_router=True):
    """dx [T, H] fp32 (the layer input's gradient) and dw_router [E, H] fp32."""
    T, H = x.shape
    E = w_router.shape[0]
    k = topk_idx.shape[1]
    dev = x.device
    _req(x, torch.bfloat16, "x")
    _req(w_router, torch.bfloat16, "w_router", (E, H))
    _req(topk_idx, torch.int32, "topk_idx", (T, k))
    _req(topk_w, torch.float32, "topk_w", (T, k))
    _req(dgate, torch.float32, "dgate", (T, k))
    _req(dxp, torch.float32, "dxp", (T * k, H))
    _req_plan(plan, T, E, k)
    _opt(dx_shared, torch.float32, "dx_shared", (T, H))
    _req(workspace, torch.uint8, "workspace")
    dx = torch.empty((T, H), dtype=torch.float32, device=dev) if dx is None else dx
    if dw_router is True:
        dw_router = torch.empty((E, H), dtype=torch.float32, device=dev)
    dw_router = None if dw_router is False else dw_router
    _req(dx, torch.float32, "dx", (T, H))
    _opt(dw_router, torch.float32, "dw_router", (E, H))
    check(lib().moe_route_backward(_p(x), _p(w_router), _p(topk_idx), _p(topk_w), _p(dgate), _p(dxp), _p(plan),
                                   _p(dx_shared), T, H, E, k, _p(dx), _p(dw_router), _p(workspace),
                                   workspace.numel(), _stream()))
    return dict(dx=dx, dw_router=dw_router)


# ---------------------------------------------------------------------------
# The 8-bit block: residual + norm, scored routing, e4m3 products
#
# These calls of a few tokens are bound by the host, so their checks, allocations and
# argument conversions are C functions (csrc/marshal.cpp): m.check(tensor, name, type,
# *shape) refuses as _req does, m.new(like, type, *shape) allocates, m.<entry point>
# takes tensors (or None) for pointers and adds the current stream, and the norm's functions
# are there as a whole.
# ---------------------------------------------------------------------------

FP8 = torch.float8_e4m3fn
SCORES = {"sigmoid": 0, "softmax": 1}
BF16_, F32_, FP8_, I32_, U8_ = range(5)              # marshal's element types
_TYPES = {torch.bfloat16: 0, torch.float32: 1}       # INVMOE_BF16, INVMOE_F32; marshal's codes too


def _type(t, name):
    """INVMOE_BF16 or INVMOE_F32 of a tensor that may be either."""
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _score(score):
    code = SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    return code


def _dims(t, name, n=2):
    s = t.shape
    if len(s) != n:
        raise ValueError(f"{name} must have {n} dimensions, got shape {tuple(s)}")
    return s


def _out(m, given, like, name, code, *shape):
    """An output: a new tensor, or the caller's (None and True mean a new one) after the usual checks."""
    if given is None or given is True:
        return m.new(like, code, *shape)
    m.check(given, name, code, *shape)
    return given


def _blocks(n):
    return (n + 127) // 128


def _plan(m, plan, T, E, k):
    m.check(plan, "plan", I32_)
    if plan.numel() < 2 * E + 1 + 2 * T * k:
        raise ValueError("plan is too small")
    return plan


def moe_router_logits(x, w_router, workspace, logits=None):
    """logits [T, E] fp32 = x @ w_router^T: moe_route_topk's router GEMM alone."""
    m = marshal()
    T, H = _dims(x, "x")
    E = w_router.shape[0]
    m.check(x, "x", BF16_, T, H)
    m.check(w_router, "w_router", BF16_, E, H)
    m.check(workspace, "workspace", U8_)
    logits = _out(m, logits, x, "logits", F32_, T, E)
    check(m.moe_router_logits(x, w_router, T, H, E, logits, workspace, workspace.numel()))
    return logits


def moe_route_select(logits, k, score="sigmoid", bias=None, n_group=1, topk_group=1, renormalize=True, scale=1.0,
                     topk_idx=None, topk_w=None, plan=None, workspace=None):
    """Experts by score (+ bias), limited to the best groups: topk_idx [T, k] int32, topk_w [T, k] fp32.

    plan: a tensor to fill, or True to allocate one (then ``workspace`` is needed): the dispatch plan."""
    m = marshal()
    T, E = _dims(logits, "logits")
    kind = _score(score)
    m.check(logits, "logits", F32_, T, E)
    if bias is not None:
        m.check(bias, "bias", F32_, E)
    topk_idx = _out(m, topk_idx, logits, "topk_idx", I32_, T, k)
    topk_w = _out(m, topk_w, logits, "topk_w", F32_, T, k)
    nbytes = 0
    if plan is not None:
        plan = m.new(logits, I32_, 2 * E + 1 + 2 * T * k) if plan is True else _plan(m, plan, T, E, k)
        m.check(workspace, "workspace", U8_)
        nbytes = workspace.numel()
    check(m.moe_route_select(logits, bias, T, E, k, kind, n_group, topk_group, bool(renormalize), scale, topk_idx,
                             topk_w, plan, workspace, nbytes))
    return {"topk_idx": topk_idx, "topk_w": topk_w, "plan": plan}


def moe_route_select_backward(logits, topk_idx, dw, score="sigmoid", renormalize=True, scale=1.0, dlogits=True,
                              dlogits_bf16=None):
    """Gradient of moe_route_select's weights: dw [T, k] fp32 -> dlogits [T, E] fp32.

    dlogits: a tensor to fill, True (allocate) or False (skip); dlogits_bf16: a bf16 tensor to fill as well."""
    m = marshal()
    T, E = _dims(logits, "logits")
    k = _dims(topk_idx, "topk_idx")[1]
    kind = _score(score)
    m.check(logits, "logits", F32_, T, E)
    m.check(topk_idx, "topk_idx", I32_, T, k)
    m.check(dw, "dw", F32_, T, k)
    dlogits = None if dlogits is False else _out(m, dlogits, logits, "dlogits", F32_, T, E)
    if dlogits_bf16 is not None:
        m.check(dlogits_bf16, "dlogits_bf16", BF16_, T, E)
    check(m.moe_route_select_backward(logits, topk_idx, dw, T, E, k, kind, bool(renormalize), scale, dlogits,
                                      dlogits_bf16))
    return dlogits


def moe_router_backward(x, w_router, dlogits_bf16, dxp, plan, k, workspace, dx_shared=None, dx=None, dw_router=True):
    """The router's part of the layer backward from dlogits_bf16 [T, E]: dx [T, H] and dw_router [E, H], fp32."""
    m = marshal()
    T, H = _dims(x, "x")
    E = w_router.shape[0]
    m.check(x, "x", BF16_, T, H)
    m.check(w_router, "w_router", BF16_, E, H)
    m.check(dlogits_bf16, "dlogits_bf16", BF16_, T, E)
    m.check(dxp, "dxp", F32_, T * k, H)
    _plan(m, plan, T, E, k)
    if dx_shared is not None:
        m.check(dx_shared, "dx_shared", F32_, T, H)
    m.check(workspace, "workspace", U8_)
    dx = _out(m, dx, x, "dx", F32_, T, H)
    dw_router = None if dw_router is False else _out(m, dw_router, x, "dw_router", F32_, E, H)
    check(m.moe_router_backward(x, w_router, dlogits_bf16, dxp, plan, dx_shared, T, H, E, k, dx, dw_router, workspace,
                                workspace.numel()))
    return dict(dx=dx, dw_router=dw_router)


def add_rms_norm(x, weight, residual=None, eps=1e-6, out=True, fp8=False, residual_out=None, q=None, scale=None,
                 rstd=None):
    """r = x + residual, normalised and scaled: dict(residual, out, q, scale, rstd).

    x [T, H] and residual [T, H] bf16 or fp32, weight [H] bf16.  ``out`` (bf16): a tensor to fill, True or False;
    ``fp8``: also the e4m3 row with a scale per 128 columns (into q and scale if given).  ``residual_out`` receives r
    in the residual's type (it may be ``residual`` itself; allocated if not given)."""
    r = marshal().norm(x, weight, residual, eps, out, fp8, residual_out, q, scale, rstd)
    return r if r.__class__ is dict else check(r)


def rms_norm_backward_workspace_size(T, H) -> int:
    return marshal().rms_norm_backward_workspace_size(T, H)


def add_rms_norm_backward(dy, x, weight, rstd, dres=None, dx=None, dweight=True, workspace=None):
    """Backward of add_rms_norm at its stored row ``x`` (its ``residual`` output, or x without one) and ``rstd``.

    dict(dx [T, H] in x's type: the gradient of that row, so of both summands; dweight [H] fp32 or None).
    dy bf16 or fp32; dres: the gradient that reaches the row from the residual stream; dx may be dres."""
    r = marshal().norm_backward(dy, x, weight, rstd, dres, dx, dweight, workspace)
    return r if r.__class__ is dict else check(r)


def fp8_quantize(x, block_rows=1, q=None, scale=None):
    """e4m3 of x [rows, cols] or [banks, rows, cols] (bf16 or fp32): (q, scale).

    block_rows 1: a scale per row and 128 columns (activations); 128: per 128 x 128 (weights)."""
    m = marshal()
    lead = tuple(x.shape[:-2])
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [rows, cols] or [banks, rows, cols], got {tuple(x.shape)}")
    xt = _type(x, "x")
    m.check(x, "x", xt)
    rows, cols = x.shape[-2:]
    banks = x.shape[0] if lead else 1
    q = _out(m, q, x, "q", FP8_, *x.shape)
    scale = _out(m, scale, x, "scale", F32_, *lead, rows if block_rows == 1 else _blocks(rows), _blocks(cols))
    check(m.fp8_quantize(x, xt, banks, rows, cols, block_rows, q, scale))
    return q, scale


def moe_permute_rows(x, plan, E, k, xp=None):
    """The bf16 rows x [T, H] in the plan's order: xp [T*k, H]."""
    m = marshal()
    T, H = _dims(x, "x")
    m.check(x, "x", BF16_, T, H)
    _plan(m, plan, T, E, k)
    xp = _out(m, xp, x, "xp", BF16_, T * k, H)
    check(m.moe_permute_rows(x, plan, T, H, E, k, xp))
    return xp


def moe_permute_fp8(q, scale, plan, E, k, xp=None, xp_scale=None):
    """The quantised rows q [T, H] and their scales in the plan's order: (xp [T*k, H], xp_scale)."""
    m = marshal()
    T, H = _dims(q, "q")
    m.check(q, "q", FP8_, T, H)
    m.check(scale, "scale", F32_, T, _blocks(H))
    _plan(m, plan, T, E, k)
    xp = _out(m, xp, q, "xp", FP8_, T * k, H)
    xp_scale = _out(m, xp_scale, q, "xp_scale", F32_, T * k, _blocks(H))
    check(m.moe_permute_fp8(q, scale, plan, T, H, E, k, xp, xp_scale))
    return xp, xp_scale


def fp8_gemm(a, a_scale, b, b_scale, workspace, out_dtype=torch.bfloat16, out=None):
    """out [M, N] = (a * a_scale) @ (b * b_scale)^T: a [M, K] e4m3 with a scale per row and 128 columns, b [N, K]
    e4m3 with a scale per 128 x 128; out bf16 or fp32."""
    m = marshal()
    M, K = _dims(a, "a")
    N = _dims(b, "b")[0]
    nb = _blocks(K)
    ot = _TYPES.get(out_dtype)
    if ot is None:
        raise ValueError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
    m.check(a, "a", FP8_, M, K)
    m.check(b, "b", FP8_, N, K)
    m.check(a_scale, "a_scale", F32_, M, nb)
    m.check(b_scale, "b_scale", F32_, _blocks(N), nb)
    m.check(workspace, "workspace", U8_)
    out = _out(m, out, a, "out", ot, M, N)
    check(m.fp8_gemm(a, a_scale, b, b_scale, M, N, K, out, ot, workspace, workspace.numel()))
    return out


def _experts_plan(m, plan, T, E, k):
    """The plan of a grouped call; None for one expert that takes every row."""
    if plan is not None:
        return _plan(m, plan, T, E, k)
    if E != 1 or k != 1:
        raise ValueError("plan may be None only for E = k = 1")
    return None


def moe_grouped_swiglu_fp8(xp, xp_scale, plan, w13, w13_scale, T, k, workspace, h=None, h_scale=None):
    """The experts' gate/up product, SwiGLU and re-quantisation: dict(h [T*k, F] e4m3, h_scale [T*k, F/128]).

    xp [T*k, H] e4m3 in plan order, w13 [E, 2F, H] e4m3 (gate rows, then up rows), w13_scale [E, 2F/128, ceil(H/128)].
    plan None: one expert (E = k = 1) for all T rows."""
    m = marshal()
    E, F2, H = _dims(w13, "w13", 3)
    if F2 % 2:
        raise ValueError(f"w13 must have an even number of rows (gate, then up), got {F2}")
    F, S, nb = F2 // 2, T * k, _blocks(H)
    m.check(xp, "xp", FP8_, S, H)
    m.check(xp_scale, "xp_scale", F32_, S, nb)
    m.check(w13, "w13", FP8_, E, F2, H)
    m.check(w13_scale, "w13_scale", F32_, E, _blocks(F2), nb)
    m.check(workspace, "workspace", U8_)
    plan = _experts_plan(m, plan, T, E, k)
    h = _out(m, h, xp, "h", FP8_, S, F)
    h_scale = _out(m, h_scale, xp, "h_scale", F32_, S, _blocks(F))
    check(m.moe_grouped_swiglu_fp8(xp, xp_scale, plan, w13, w13_scale, T, H, E, k, F, h, h_scale, workspace,
                                   workspace.numel()))
    return {"h": h, "h_scale": h_scale}


def moe_grouped_down_fp8(h, h_scale, plan, w2, w2_scale, T, k, workspace, y=None):
    """The experts' down product: y [T*k, H] fp32.  h [T*k, F] e4m3, w2 [E, H, F] e4m3, w2_scale
    [E, ceil(H/128), F/128]; plan None: one expert (E = k = 1) for all T rows."""
    m = marshal()
    E, H, F = _dims(w2, "w2", 3)
    S, nb = T * k, _blocks(F)
    m.check(h, "h", FP8_, S, F)
    m.check(h_scale, "h_scale", F32_, S, nb)
    m.check(w2, "w2", FP8_, E, H, F)
    m.check(w2_scale, "w2_scale", F32_, E, _blocks(H), nb)
    m.check(workspace, "workspace", U8_)
    plan = _experts_plan(m, plan, T, E, k)
    y = _out(m, y, h, "y", F32_, S, H)
    check(m.moe_grouped_down_fp8(h, h_scale, plan, w2, w2_scale, T, H, E, k, F, y, workspace, workspace.numel()))
    return y


# ---------------------------------------------------------------------------
# A drafted decode step: the layer of a few tokens in one kernel, norms around a block, verification of drafted tokens
# ---------------------------------------------------------------------------

DECODE_MAX_TOKENS, DECODE_MAX_EXPERTS = 16, 512      # of moe_layer_decode


def moe_decode_workspace_size(T, H, E, k, F, F_shared=0) -> int:
    return int(lib().moe_decode_workspace_size(T, H, E, k, F, F_shared))


def moe_layer_decode(x, w_router, w13, w2, k, workspace, ws13=None, ws2=None, score=None, bias=None, n_group=1, topk_group=1,
                     renormalize=True, scale=1.0, out=True, out_bf16=None, logits=None, topk_idx=None, topk_w=None):
    """The whole layer of at most 16 tokens in one kernel, with moe_layer_forward's bits:
    dict(out, out_bf16, logits, topk_idx, topk_w).

    score None: the softmax over the k largest logits; "sigmoid" or "softmax": the choice of moe_route_select, with its
    arguments.  out [T, H] fp32 and out_bf16: a tensor to fill, True, or False / None to skip it (not both).
    workspace: at least moe_decode_workspace_size bytes from new_workspace."""
    m = marshal()
    T, H = _dims(x, "x")
    E, F2, _ = _dims(w13, "w13", 3)
    F, Fs = F2 // 2, 0
    kind = 2 if score is None else _score(score)
    if (ws13 is None) != (ws2 is None):
        raise ValueError("ws13 and ws2 go together")
    m.check(x, "x", BF16_, T, H)
    m.check(w_router, "w_router", BF16_, E, H)
    m.check(w13, "w13", BF16_, E, 2 * F, H)
    m.check(w2, "w2", BF16_, E, H, F)
    if ws13 is not None:
        Fs = _dims(ws13, "ws13")[0] // 2
        m.check(ws13, "ws13", BF16_, 2 * Fs, H)
        m.check(ws2, "ws2", BF16_, H, Fs)
    if bias is not None:
        m.check(bias, "bias", F32_, E)
    m.check(workspace, "workspace", U8_)
    out = None if out is False else _out(m, out, x, "out", F32_, T, H)
    out_bf16 = None if out_bf16 is None or out_bf16 is False else _out(m, out_bf16, x, "out_bf16", BF16_, T, H)
    logits = _out(m, logits, x, "logits", F32_, T, E)
    topk_idx = _out(m, topk_idx, x, "topk_idx", I32_, T, k)
    topk_w = _out(m, topk_w, x, "topk_w", F32_, T, k)
    check(m.moe_layer_decode(x, w_router, w13, w2, ws13, ws2, T, H, E, k, F, Fs, kind, bias, n_group, topk_group,
                             bool(renormalize), scale, out, out_bf16, logits, topk_idx, topk_w, workspace,
                             workspace.numel()))
    return {"out": out, "out_bf16": out_bf16, "logits": logits, "topk_idx": topk_idx, "topk_w": topk_w}


def sandwich_norm(x, w_post, residual, w_next=None, gate=None, residual_scale=1.0, branch_scale=1.0, eps=1e-6, out=True,
                  fp8=False, residual_out=None, q=None, scale=None, rstd_post=None, rstd=None):
    """The norms after and before a block: dict(residual, out, q, scale, rstd_post, rstd).

    residual = residual_scale * residual + branch_scale * gate * rms_norm(x) * w_post, stored in the residual's type (into
    ``residual_out``, which may be ``residual`` itself); out = rms_norm(residual) * w_next in bf16 (a tensor to fill, True or
    False), with ``fp8`` also as the e4m3 row with a scale per 128 columns.  Without w_next there is no second norm.
    x, residual [T, H] bf16 or fp32; weights [H] bf16; gate None, [H] bf16 (a channel's) or [T] fp32 (a token's)."""
    r = marshal().sandwich(x, w_post, residual, w_next, gate, residual_scale, branch_scale, eps, out, fp8, residual_out, q,
                           scale, rstd_post, rstd)
    return r if r.__class__ is dict else check(r)


def sandwich_norm_backward_workspace_size(T, H) -> int:
    return int(lib().sandwich_norm_backward_workspace_size(T, H))


def sandwich_norm_backward(dy, dres, x, w_post, rstd_post, residual, w_next=None, rstd=None, gate=None, residual_scale=1.0,
                           branch_scale=1.0, dx=None, dresidual=None, dweights=True, workspace=None):
    """Backward of sandwich_norm at its x, its stored row (``residual`` here: its ``residual`` output) and its rstd_post and
    rstd: dict(dx, dresidual, dw_post, dw_next, dgate).

    dy [T, H] bf16 or fp32: the gradient of ``out`` (None without w_next); dres [T, H] in the residual's type: the gradient
    that reaches the stored row from the residual stream (None: none).  dx has x's type, dresidual the residual's; the
    weights' gradients are fp32 [H] (skipped with dweights=False), dgate [H] or [T] fp32 as the gate.  ``workspace``:
    sandwich_norm_backward_workspace_size bytes, whose status check_status reads (allocated and dropped if not given).  Where a
    kernel gives up waiting, what depends on the rows it waited for is NaN."""
    r = marshal().sandwich_backward(dy, dres, x, w_post, rstd_post, residual, w_next, rstd, gate, residual_scale, branch_scale,
                                    dx, dresidual, dweights, workspace)
    return r if r.__class__ is dict else check(r)


def verify_workspace_size(B, D, V) -> int:
    return int(lib().verify_workspace_size(B, D, V))


def verify_drafts(logits, noise, workspace, draft_tokens=None, draft_logits=None, accept_u=None, n_draft=None,
                  temperature=1.0, tokens=None, n_accepted=None, logp=None):
    """Accept each request's drafts against the target's probabilities and draw the token that follows:
    dict(tokens [B, D+1] int32, n_accepted [B] int32, logp [B, D+1] fp32).

    logits [B, D+1, V] bf16 or fp32 of the target; draft_tokens [B, D] int32 with their draft_logits [B, D, V] (None: a
    drafter without probabilities) and accept_u [B, D] fp32 uniform in [0, 1); n_draft [B] int32: how many of the D count
    (None: all); noise [B, V] fp32 exponential.  temperature: a number or [B] fp32, 0 for greedy.  Without draft_tokens one
    token per request is drawn.  tokens: the accepted drafts, the drawn token, -1 behind it; logp: of those tokens, 0 behind.
    workspace: at least verify_workspace_size(B, D, V) bytes, any content."""
    r = marshal().verify(logits, noise, workspace, draft_tokens, draft_logits, accept_u, n_draft, temperature, tokens,
                         n_accepted, logp)
    return r if r.__class__ is dict else check(r)


def gemm_bf16(a, b, workspace, variant=0, out=None):
    """Diagnostic: the dense tcgen05 GEMM engine alone, d = a @ b^T in fp32.

    variant 5 takes b as [K, N] (d = a @ b); variant 6 takes a as [K, M] and b as
    [K, N] (d = a^T @ b)."""
    v = int(variant) & 0xff
    if v == 6:
        K, M = a.shape
    else:
        M, K = a.shape
    N = b.shape[1] if v in (5, 6) else b.shape[0]
    _req(a, torch.bfloat16, "a")
    _req(b, torch.bfloat16, "b", (K, N) if v in (5, 6) else (N, K))
    out = torch.empty((M, N), dtype=torch.float32, device=a.device) if out is None else out
    _req(out, torch.float32, "out", (M, N))
    check(lib().invmoe_gemm_bf16(_p(a), _p(b), M, N, K, _p(out), int(variant), _p(workspace), workspace.numel(),
                                 _stream()))
    return out


def debug_timeout_probe(workspace, timeout_us=20000):
    check(lib().invmoe_debug_timeout_probe(_p(workspace), workspace.numel(), int(timeout_us), _stream()))


def debug_stalled_backward(dy, dres, x, w_post, rstd_post, residual, w_next, rstd, group, workspace, timeout_us=20000):
    """sandwich_norm_backward (all fp32, no gate, H <= 2048) whose blocks wait in vain for a group of their second row."""
    T, H = x.shape
    for t in (dy, dres, x, residual):
        if t is not None:
            _req(t, torch.float32, "rows", (T, H))
    dx, dresidual = torch.empty_like(x), torch.empty_like(x)
    dw_post = torch.empty(H, dtype=torch.float32, device=x.device)
    dw_next = None if dy is None else torch.empty_like(dw_post)
    check(lib().invmoe_debug_stalled_backward(_p(dy), _p(dres), _p(x), _p(w_post), _p(rstd_post), _p(residual), _p(w_next),
                                              _p(rstd), T, H, int(group), int(timeout_us), _p(dx), _p(dresidual), _p(dw_post),
                                              _p(dw_next), _p(workspace), workspace.numel(), _stream()))
    return dict(dx=dx, dresidual=dresidual, dw_post=dw_post, dw_next=dw_next)
