// api_step.cu -- the extern "C" entry points of a drafted decode step: the layer of a few tokens, norms around a
// block, drafted tokens.
#include <cuda_runtime.h>

#include "checks.h"
#include "fp8.cuh"
#include "internal.h"

using namespace invmoe;

namespace {

int check_rows(int T, int H, int x_type, int residual_type, const void* gate, int gate_kind, float residual_scale,
               float branch_scale) {
  REQUIRE(x_type == INVMOE_BF16 || x_type == INVMOE_F32, INVMOE_ERR_INVALID_ARG, "x_type must be INVMOE_BF16 or INVMOE_F32");
  REQUIRE(residual_type == INVMOE_BF16 || residual_type == INVMOE_F32, INVMOE_ERR_INVALID_ARG,
          "residual_type must be INVMOE_BF16 or INVMOE_F32");
  REQUIRE(T >= 0 && H > 0, INVMOE_ERR_INVALID_ARG, "need T >= 0, H > 0");
  REQUIRE(H % 16 == 0 && H <= 32768, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 16 up to 32768", H);
  REQUIRE(gate_kind == INVMOE_GATE_NONE || gate_kind == INVMOE_GATE_CHANNEL || gate_kind == INVMOE_GATE_TOKEN,
          INVMOE_ERR_INVALID_ARG, "gate_kind must be INVMOE_GATE_NONE, INVMOE_GATE_CHANNEL or INVMOE_GATE_TOKEN");
  REQUIRE((gate == nullptr) == (gate_kind == INVMOE_GATE_NONE) || T == 0, INVMOE_ERR_INVALID_ARG,
          "gate and gate_kind do not go together");
  REQUIRE(residual_scale == residual_scale && branch_scale == branch_scale, INVMOE_ERR_INVALID_ARG, "a scale is NaN");
  return INVMOE_OK;
}

size_t matrix_bytes(int T, int H, int type) { return static_cast<size_t>(T) * H * (type == INVMOE_F32 ? 4 : 2); }

// An array's addresses; none of an absent or empty one.
struct Span {
  uintptr_t lo = 0, hi = 0;
  Span(const void* at, size_t bytes) {
    if (at != nullptr && bytes != 0) {
      lo = reinterpret_cast<uintptr_t>(at);
      hi = lo + bytes;
    }
  }
};
// No output has a byte in common with an input or with another output.  (Without a branch per pair: a call of a few rows is
// bound by the host.)
template <size_t OUT, size_t IN>
bool outputs_apart(const Span (&outs)[OUT], const Span (&ins)[IN]) {
  bool meet = false;
  for (size_t i = 0; i < OUT; ++i) {
    for (size_t j = 0; j < IN; ++j) meet |= (outs[i].lo < ins[j].hi) & (ins[j].lo < outs[i].hi);
    for (size_t j = 0; j < i; ++j) meet |= (outs[i].lo < outs[j].hi) & (outs[j].lo < outs[i].hi);
  }
  return !meet;
}

// moe_layer_decode's part of the workspace behind the status block: offsets of its arrays.
struct DecodeScratch {
  size_t logits, h, hs, y, ys, total;
};
DecodeScratch decode_scratch(int T, int H, int E, int k, int F, int F_shared) {
  DecodeScratch s{};
  const size_t rows = static_cast<size_t>(T) * k;
  s.logits = align_up(kDecodeFlags * sizeof(int), 256);
  s.h = s.logits + align_up(static_cast<size_t>(T) * E * 4, 256);
  s.hs = s.h + align_up(rows * F * 2, 256);
  s.y = s.hs + align_up(static_cast<size_t>(T) * F_shared * 2, 256);
  s.ys = s.y + align_up(rows * H * 4, 256);
  s.total = s.ys + (F_shared > 0 ? align_up(static_cast<size_t>(T) * H * 4, 256) : 0);
  return s;
}

}  // namespace

extern "C" {

int sandwich_norm(const void* x, int x_type, const void* w_post, const void* residual, int residual_type, const void* gate,
                  int gate_kind, const void* w_next, int T, int H, float residual_scale, float branch_scale, float eps,
                  void* residual_out, void* out, void* q, float* scale, float* rstd_post, float* rstd, void* stream) {
  const int rc = check_rows(T, H, x_type, residual_type, gate, gate_kind, residual_scale, branch_scale);
  if (rc) return rc;
  REQUIRE(eps >= 0.0f, INVMOE_ERR_INVALID_ARG, "need eps >= 0");
  REQUIRE((q == nullptr) == (scale == nullptr), INVMOE_ERR_INVALID_ARG, "q and scale go together");
  if (T == 0) return INVMOE_OK;
  REQUIRE((w_next != nullptr) == (out != nullptr || q != nullptr), INVMOE_ERR_INVALID_ARG,
          "w_next goes with an output of the second norm (out, q)");
  REQUIRE(w_next != nullptr || rstd == nullptr, INVMOE_ERR_INVALID_ARG, "rstd without w_next");
  REQUIRE_PTR(x); REQUIRE_PTR(w_post); REQUIRE_PTR(residual); REQUIRE_PTR(residual_out);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_post); REQUIRE_ALIGNED(residual); REQUIRE_ALIGNED(residual_out);
  REQUIRE_ALIGNED(w_next); REQUIRE_ALIGNED(out); REQUIRE_ALIGNED(q);
  if (gate_kind == INVMOE_GATE_CHANNEL) REQUIRE_ALIGNED(gate);
  const size_t xn = matrix_bytes(T, H, x_type), rn = matrix_bytes(T, H, residual_type), on = matrix_bytes(T, H, INVMOE_BF16);
  REQUIRE(same_or_apart(residual_out, residual, rn), INVMOE_ERR_INVALID_ARG,
          "residual_out overlaps residual without being it");
  const size_t each = static_cast<size_t>(T) * 4, row = static_cast<size_t>(H) * 2;
  const Span ins[] = {{x, xn}, {w_post, row}, {w_next, row}, {gate, gate_kind == INVMOE_GATE_CHANNEL ? row : each},
                      {residual_out == residual ? nullptr : residual, rn}};
  const Span outs[] = {{residual_out, rn}, {out, on}, {q, on / 2}, {scale, each * ((H + kFp8Block - 1) / kFp8Block)},
                       {rstd_post, each}, {rstd, each}};
  REQUIRE(outputs_apart(outs, ins), INVMOE_ERR_INVALID_ARG, "an output overlaps another one or an input");
  return sandwich_launch({x, x_type == INVMOE_F32, w_post, residual, residual_type == INVMOE_F32, gate, gate_kind, w_next, T,
                          H, residual_scale, branch_scale, eps, residual_out, out, q, scale, rstd_post, rstd},
                         static_cast<cudaStream_t>(stream));
}

size_t sandwich_norm_backward_workspace_size(int T, int H) {
  if (T <= 0 || H <= 0) return kStatusBytes;
  return kStatusBytes + align_up(T, 64) * sizeof(float) +
         align_up(static_cast<size_t>(sandwich_bwd_plan(T, H).parts) * 2 * H * sizeof(float), 256);
}

int sandwich_norm_backward(const void* dy, int dy_type, const void* dres, const void* x, int x_type, const void* w_post,
                           const float* rstd_post, const void* residual, int residual_type, const void* w_next,
                           const float* rstd, const void* gate, int gate_kind, int T, int H, float residual_scale,
                           float branch_scale, void* dx, void* dresidual, float* dw_post, float* dw_next, float* dgate,
                           void* workspace, size_t ws_bytes, void* stream) {
  const int rc = check_rows(T, H, x_type, residual_type, gate, gate_kind, residual_scale, branch_scale);
  if (rc) return rc;
  REQUIRE(dy_type == INVMOE_BF16 || dy_type == INVMOE_F32, INVMOE_ERR_INVALID_ARG,
          "dy_type must be INVMOE_BF16 or INVMOE_F32");
  const bool channel = gate_kind == INVMOE_GATE_CHANNEL;
  REQUIRE(dw_post != nullptr || (dw_next == nullptr && (dgate == nullptr || !channel)), INVMOE_ERR_INVALID_ARG,
          "dw_next and a channel gate's dgate come with dw_post");
  REQUIRE(dw_next == nullptr || w_next != nullptr || T == 0, INVMOE_ERR_INVALID_ARG, "dw_next without w_next");
  REQUIRE(dgate == nullptr || gate_kind != INVMOE_GATE_NONE, INVMOE_ERR_INVALID_ARG, "dgate without a gate");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    for (float* g : {dw_post, dw_next, channel ? dgate : nullptr}) {
      if (g == nullptr) continue;
      const int e = check_cuda(cudaMemsetAsync(g, 0, static_cast<size_t>(H) * sizeof(float), st), "cudaMemsetAsync");
      if (e) return e;
    }
    return INVMOE_OK;
  }
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= sandwich_norm_backward_workspace_size(T, H), INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  REQUIRE((dy != nullptr) == (w_next != nullptr) && (dy != nullptr) == (rstd != nullptr), INVMOE_ERR_INVALID_ARG,
          "dy, w_next and rstd go together");
  REQUIRE(dy != nullptr || dres != nullptr, INVMOE_ERR_INVALID_ARG, "dy and dres are both NULL");
  REQUIRE(dy == nullptr || residual != nullptr, INVMOE_ERR_INVALID_ARG, "residual is NULL");
  REQUIRE_PTR(x); REQUIRE_PTR(w_post); REQUIRE_PTR(rstd_post); REQUIRE_PTR(dx); REQUIRE_PTR(dresidual);
  REQUIRE_ALIGNED(dy); REQUIRE_ALIGNED(dres); REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_post); REQUIRE_ALIGNED(residual);
  REQUIRE_ALIGNED(w_next); REQUIRE_ALIGNED(dx); REQUIRE_ALIGNED(dresidual); REQUIRE_ALIGNED(workspace);
  if (channel) REQUIRE_ALIGNED(gate);
  const size_t xn = matrix_bytes(T, H, x_type), rn = matrix_bytes(T, H, residual_type), yn = matrix_bytes(T, H, dy_type);
  const size_t each = static_cast<size_t>(T) * 4, row = static_cast<size_t>(H) * 2;
  const Span ins[] = {{x, xn}, {dy, yn}, {dres, rn}, {dy != nullptr ? residual : nullptr, rn}, {w_post, row}, {w_next, row},
                      {rstd_post, each}, {rstd, each}, {gate, channel ? row : each}};
  const Span outs[] = {{dx, xn}, {dresidual, rn}, {dw_post, 2 * row}, {dw_next, 2 * row}, {dgate, channel ? 2 * row : each}};
  REQUIRE(outputs_apart(outs, ins), INVMOE_ERR_INVALID_ARG, "an output overlaps another one or an input");
  return sandwich_bwd_launch(
      {dy, dy_type == INVMOE_F32, dres, x, x_type == INVMOE_F32, w_post, rstd_post, residual, residual_type == INVMOE_F32,
       w_next, rstd, gate, gate_kind, T, H, residual_scale, branch_scale, dx, dresidual, dw_post, dw_next, dgate,
       reinterpret_cast<float*>(scratch(workspace)), status_word(workspace)},
      st);
}

int invmoe_debug_stalled_backward(const float* dy, const float* dres, const float* x, const void* w_post,
                                  const float* rstd_post, const float* residual, const void* w_next, const float* rstd,
                                  int T, int H, int group, int timeout_us, float* dx, float* dresidual, float* dw_post,
                                  float* dw_next, void* workspace, size_t ws_bytes, void* stream) {
  const int rc = check_rows(T, H, INVMOE_F32, INVMOE_F32, nullptr, INVMOE_GATE_NONE, 1.0f, 1.0f);
  if (rc) return rc;
  REQUIRE(T > 0 && H <= 2048, INVMOE_ERR_UNSUPPORTED_SHAPE, "need T > 0 and H <= 2048");
  REQUIRE(group == 0 || group == 1, INVMOE_ERR_INVALID_ARG, "group must be 0 or 1");
  REQUIRE(timeout_us >= 1 && timeout_us <= 2000000, INVMOE_ERR_INVALID_ARG, "timeout_us must be 1..2000000");
  const bool next = dy != nullptr;
  REQUIRE(next == (w_next != nullptr) && next == (rstd != nullptr) && next == (dw_next != nullptr), INVMOE_ERR_INVALID_ARG,
          "dy, w_next, rstd and dw_next go together");
  REQUIRE(dy == nullptr || residual != nullptr, INVMOE_ERR_INVALID_ARG, "residual is NULL");
  REQUIRE_PTR(dres); REQUIRE_PTR(x); REQUIRE_PTR(w_post); REQUIRE_PTR(rstd_post); REQUIRE_PTR(dx); REQUIRE_PTR(dresidual);
  REQUIRE_PTR(dw_post); REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= sandwich_norm_backward_workspace_size(T, H), INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  REQUIRE_ALIGNED(dy); REQUIRE_ALIGNED(dres); REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_post); REQUIRE_ALIGNED(residual);
  REQUIRE_ALIGNED(w_next); REQUIRE_ALIGNED(dx); REQUIRE_ALIGNED(dresidual); REQUIRE_ALIGNED(workspace);
  SandwichBwdCall c{dy, true, dres, x, true, w_post, rstd_post, residual, true, w_next, rstd, nullptr, INVMOE_GATE_NONE, T, H,
                    1.0f, 1.0f, dx, dresidual, dw_post, dw_next, nullptr, reinterpret_cast<float*>(scratch(workspace)),
                    status_word(workspace)};
  c.stalled_ns = static_cast<unsigned long long>(timeout_us) * 1000ull;
  c.stalled = group;
  return sandwich_bwd_launch(c, static_cast<cudaStream_t>(stream));
}

size_t moe_decode_workspace_size(int T, int H, int E, int k, int F, int F_shared) {
  if (T <= 0 || T > kDecodeMaxTokens || H <= 0 || E <= 0 || k <= 0 || k > 32 || F <= 0 || F_shared < 0) return kStatusBytes;
  return kStatusBytes + decode_scratch(T, H, E, k, F, F_shared).total;
}

int moe_layer_decode(const void* x, const void* w_router, const void* w13, const void* w2, const void* ws13, const void* ws2,
                     int T, int H, int E, int k, int F, int F_shared, int score, const float* bias, int n_group,
                     int topk_group, int renormalize, float scale, float* out, void* out_bf16, float* logits,
                     int32_t* topk_idx, float* topk_w, void* workspace, size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0 && H > 0 && E > 0 && k > 0 && F > 0 && F_shared >= 0, INVMOE_ERR_INVALID_ARG,
          "need T, F_shared >= 0 and H, E, k, F > 0");
  REQUIRE(T <= kDecodeMaxTokens, INVMOE_ERR_UNSUPPORTED_SHAPE, "T=%d > %d", T, kDecodeMaxTokens);
  REQUIRE(E <= kDecodeMaxExperts, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d > %d", E, kDecodeMaxExperts);
  REQUIRE(k <= E, INVMOE_ERR_INVALID_ARG, "k=%d must satisfy 1 <= k <= E=%d", k, E);
  REQUIRE(k <= 32, INVMOE_ERR_UNSUPPORTED_SHAPE, "k=%d > 32", k);
  REQUIRE(H % 64 == 0 && H <= 64 * kDecodeMaxBlocks, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 64 up to %d", H,
          64 * kDecodeMaxBlocks);
  REQUIRE(F % 64 == 0 && F <= 1 << 20, INVMOE_ERR_UNSUPPORTED_SHAPE, "F=%d is not a multiple of 64 up to 2^20", F);
  REQUIRE(F_shared % 64 == 0 && F_shared <= 1 << 20, INVMOE_ERR_UNSUPPORTED_SHAPE,
          "F_shared=%d is not a multiple of 64 up to 2^20", F_shared);
  REQUIRE(score == INVMOE_SCORE_TOPK || score == INVMOE_SCORE_SIGMOID || score == INVMOE_SCORE_SOFTMAX,
          INVMOE_ERR_INVALID_ARG, "score must be INVMOE_SCORE_TOPK, INVMOE_SCORE_SIGMOID or INVMOE_SCORE_SOFTMAX");
  if (score == INVMOE_SCORE_TOPK) {
    REQUIRE(bias == nullptr && n_group == 1 && topk_group == 1 && scale == 1.0f && renormalize, INVMOE_ERR_INVALID_ARG,
            "bias, groups, scale and plain weights need a score");
  } else {
    REQUIRE(n_group >= 1 && n_group <= 32 && E % n_group == 0, INVMOE_ERR_INVALID_ARG,
            "n_group=%d must be 1..32 and divide E=%d", n_group, E);
    REQUIRE(topk_group >= 1 && topk_group <= n_group, INVMOE_ERR_INVALID_ARG, "topk_group=%d must be 1..n_group=%d",
            topk_group, n_group);
    REQUIRE(k <= E / n_group * topk_group, INVMOE_ERR_INVALID_ARG, "k=%d exceeds the %d experts of %d groups", k,
            E / n_group * topk_group, topk_group);
  }
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= moe_decode_workspace_size(T, H, E, k, F, F_shared), INVMOE_ERR_WORKSPACE_TOO_SMALL,
          "workspace too small");
  REQUIRE_PTR(x); REQUIRE_PTR(w_router); REQUIRE_PTR(w13); REQUIRE_PTR(w2);
  REQUIRE(out != nullptr || out_bf16 != nullptr, INVMOE_ERR_INVALID_ARG, "out and out_bf16 are both NULL");
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_router); REQUIRE_ALIGNED(w13); REQUIRE_ALIGNED(w2);
  REQUIRE_ALIGNED(out); REQUIRE_ALIGNED(out_bf16); REQUIRE_ALIGNED(workspace);
  if (F_shared > 0) {
    REQUIRE_PTR(ws13); REQUIRE_PTR(ws2);
    REQUIRE_ALIGNED(ws13); REQUIRE_ALIGNED(ws2);
  }
  // columns of x are read until the last block is done with its gate/up units, long after others have written outputs
  // (and the logits while other blocks already combine)
  const size_t xn = matrix_bytes(T, H, INVMOE_BF16), pairs = static_cast<size_t>(T) * k * 4;
  const Span ins[] = {{x, xn}};
  const Span outs[] = {{out, 2 * xn}, {out_bf16, xn}, {logits, static_cast<size_t>(T) * E * 4}, {topk_idx, pairs},
                       {topk_w, pairs}};
  REQUIRE(outputs_apart(outs, ins), INVMOE_ERR_INVALID_ARG, "an output overlaps x or another one");
  const DecodeScratch s = decode_scratch(T, H, E, k, F, F_shared);
  uint8_t* base = scratch(workspace);
  DecodeParams p{};
  p.T = T; p.H = H; p.E = E; p.k = k; p.F = F; p.Fs = F_shared;
  p.score = score == INVMOE_SCORE_TOPK ? kDecodeTopk : score == INVMOE_SCORE_SIGMOID ? kDecodeSigmoid : kDecodeSoftmax;
  p.bias = bias;
  p.n_group = n_group;
  p.topk_group = topk_group;
  p.renorm = renormalize != 0;
  p.scale = scale;
  p.logits = logits != nullptr ? logits : reinterpret_cast<float*>(base + s.logits);
  p.topk_idx = topk_idx;
  p.topk_w = topk_w;
  p.h = reinterpret_cast<__nv_bfloat16*>(base + s.h);
  p.hs = reinterpret_cast<__nv_bfloat16*>(base + s.hs);
  p.y = reinterpret_cast<float*>(base + s.y);
  p.ys = reinterpret_cast<float*>(base + s.ys);
  p.out = out;
  p.out_bf16 = static_cast<__nv_bfloat16*>(out_bf16);
  p.status = status_word(workspace);
  p.ctl = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + 192);
  p.flags = reinterpret_cast<int*>(base);
  p.timeout_ns = kTimeoutNs;
  return moe_decode_launch({x, w_router, w13, w2, ws13, ws2}, p, static_cast<cudaStream_t>(stream));
}

size_t verify_workspace_size(int B, int D, int V) {
  if (B <= 0 || D < 0 || V <= 0) return kStatusBytes;
  const size_t chunks = verify_chunks(V);
  return kStatusBytes + align_up(static_cast<size_t>(B) * sizeof(int32_t), 256) +
         align_up(static_cast<size_t>(B) * verify_race_chunks(V) * sizeof(unsigned long long), 256) +
         static_cast<size_t>(B) * (2 * static_cast<size_t>(D) + 1) * chunks * 16;
}

int verify_drafts(const void* logits, int logits_type, const void* draft_logits, const int32_t* draft_tokens,
                  const float* accept_u, const float* noise, const int32_t* n_draft, const float* temperature, float tau,
                  int B, int D, int V, int32_t* tokens, int32_t* n_accepted, float* logp, void* workspace, size_t ws_bytes,
                  void* stream) {
  REQUIRE(logits_type == INVMOE_BF16 || logits_type == INVMOE_F32, INVMOE_ERR_INVALID_ARG,
          "logits_type must be INVMOE_BF16 or INVMOE_F32");
  REQUIRE(B >= 0 && D >= 0 && V > 0, INVMOE_ERR_INVALID_ARG, "need B, D >= 0 and V > 0");
  REQUIRE(D <= kVerifyMaxDrafts, INVMOE_ERR_UNSUPPORTED_SHAPE, "D=%d > %d", D, kVerifyMaxDrafts);
  // columns are counted in 32 bits, up to a chunk past the last
  REQUIRE(V <= 1 << 30, INVMOE_ERR_UNSUPPORTED_SHAPE, "V=%d > 2^30", V);
  REQUIRE(temperature != nullptr || tau >= 0.0f, INVMOE_ERR_INVALID_ARG, "need a temperature >= 0");
  const int chunks = verify_chunks(V), rows = D + 1 + (draft_logits != nullptr ? D : 0);
  REQUIRE(static_cast<long long>(B) * rows <= 0x7fffffffLL / chunks && B <= 0x3fffffff / verify_race_chunks(V),
          INVMOE_ERR_UNSUPPORTED_SHAPE,
          "too many rows for one launch");
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= verify_workspace_size(B, D, V), INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  REQUIRE_ALIGNED(workspace);
  if (B == 0) return INVMOE_OK;
  REQUIRE_PTR(logits); REQUIRE_PTR(noise); REQUIRE_PTR(tokens); REQUIRE_PTR(n_accepted); REQUIRE_PTR(logp);
  REQUIRE(D > 0 || draft_logits == nullptr, INVMOE_ERR_INVALID_ARG, "draft_logits without drafts");
  if (D > 0) { REQUIRE_PTR(draft_tokens); REQUIRE_PTR(accept_u); }
  REQUIRE_ALIGNED(logits); REQUIRE_ALIGNED(draft_logits); REQUIRE_ALIGNED(noise);
  // a request's outputs are written while others are still being read
  const size_t each = static_cast<size_t>(B) * 4, wide = each * V, row = wide / (logits_type == INVMOE_F32 ? 1 : 2);
  const Span ins[] = {{logits, row * (D + 1)}, {draft_logits, row * D}, {draft_tokens, each * D}, {accept_u, each * D},
                      {noise, wide},           {n_draft, each},         {temperature, each}};
  const Span outs[] = {{tokens, each * (D + 1)}, {n_accepted, each}, {logp, each * (D + 1)}};
  REQUIRE(outputs_apart(outs, ins), INVMOE_ERR_INVALID_ARG, "an output overlaps an input or another one");
  uint8_t* s = scratch(workspace);
  VerifyCall c{logits, draft_logits, draft_tokens, accept_u, noise, n_draft, temperature, tau, B, D, V, rows, chunks,
               tokens, n_accepted, logp, reinterpret_cast<int32_t*>(s), nullptr, nullptr};
  s += align_up(static_cast<size_t>(B) * sizeof(int32_t), 256);
  c.racers = s;
  c.stats = s + align_up(static_cast<size_t>(B) * verify_race_chunks(V) * sizeof(unsigned long long), 256);
  return verify_launch(c, logits_type == INVMOE_F32, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
