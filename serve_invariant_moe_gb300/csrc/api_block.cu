// api_block.cu -- the extern "C" entry points of the 8-bit block: scored routing, norm, e4m3 products.
#include <cuda_runtime.h>

#include "checks.h"
#include "fp8.cuh"
#include "internal.h"

using namespace invmoe;

namespace {

int check_select(int T, int E, int k, int score, int n_group, int topk_group) {
  REQUIRE(T >= 0 && E > 0 && k > 0, INVMOE_ERR_INVALID_ARG, "need T >= 0, E, k > 0");
  REQUIRE(score == INVMOE_SCORE_SIGMOID || score == INVMOE_SCORE_SOFTMAX, INVMOE_ERR_INVALID_ARG,
          "score must be INVMOE_SCORE_SIGMOID or INVMOE_SCORE_SOFTMAX");
  REQUIRE(E <= 1024, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d > 1024", E);
  REQUIRE(k <= 32, INVMOE_ERR_UNSUPPORTED_SHAPE, "k=%d > 32", k);
  REQUIRE(n_group >= 1 && n_group <= 32 && E % n_group == 0, INVMOE_ERR_INVALID_ARG,
          "n_group=%d must be 1..32 and divide E=%d", n_group, E);
  REQUIRE(topk_group >= 1 && topk_group <= n_group, INVMOE_ERR_INVALID_ARG, "topk_group=%d must be 1..n_group=%d",
          topk_group, n_group);
  REQUIRE(k <= E / n_group * topk_group, INVMOE_ERR_INVALID_ARG, "k=%d exceeds the %d experts of %d groups", k,
          E / n_group * topk_group, topk_group);
  return INVMOE_OK;
}

int check_type(int type, const char* what) {
  REQUIRE(type == INVMOE_BF16 || type == INVMOE_F32, INVMOE_ERR_INVALID_ARG, "%s must be INVMOE_BF16 or INVMOE_F32", what);
  return INVMOE_OK;
}

size_t matrix_bytes(int T, int H, int type) { return static_cast<size_t>(T) * H * (type == INVMOE_F32 ? 4 : 2); }

int check_width(int H) {
  REQUIRE(H > 0, INVMOE_ERR_INVALID_ARG, "need H > 0");
  REQUIRE(H % 16 == 0 && H <= 32768, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 16 up to 32768", H);
  return INVMOE_OK;
}

int check_grouped(int T, int H, int E, int k, int F) {
  REQUIRE(T >= 0 && H > 0 && E > 0 && k > 0 && F > 0, INVMOE_ERR_INVALID_ARG, "need T >= 0, H, E, k, F > 0");
  REQUIRE(E <= 1024, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d > 1024", E);
  REQUIRE(H % 16 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 16", H);
  REQUIRE(F % 128 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "F=%d is not a multiple of 128", F);
  REQUIRE(static_cast<long long>(T) * k <= 0x7fffffffLL, INVMOE_ERR_UNSUPPORTED_SHAPE, "T * k exceeds 2^31 - 1");
  REQUIRE(2LL * F * E <= 0x7fffff00LL && static_cast<long long>(H) * E <= 0x7fffff00LL, INVMOE_ERR_UNSUPPORTED_SHAPE,
          "too many weight rows");
  return INVMOE_OK;
}

}  // namespace

extern "C" {

int moe_router_logits(const void* x, const void* w_router, int T, int H, int E, float* logits, void* workspace,
                      size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0 && H > 0 && E > 0, INVMOE_ERR_INVALID_ARG, "need T >= 0, H, E > 0");
  REQUIRE(E <= 1024, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d > 1024", E);
  REQUIRE(H % 64 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 64", H);
  REQUIRE(E % 4 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d is not a multiple of 4", E);
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= kStatusBytes, INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(w_router); REQUIRE_PTR(logits);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_router); REQUIRE_ALIGNED(logits); REQUIRE_ALIGNED(workspace);
  return router_gemm_run(x, w_router, T, H, E, logits, status_word(workspace), static_cast<cudaStream_t>(stream));
}

int moe_route_select(const float* logits, const float* bias, int T, int E, int k, int score, int n_group,
                     int topk_group, int renormalize, float scale, int32_t* topk_idx, float* topk_w, int32_t* plan,
                     void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_select(T, E, k, score, n_group, topk_group);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (plan != nullptr) {
    REQUIRE_PTR(workspace);
    REQUIRE(ws_bytes >= kStatusBytes + route_ws(T, E), INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
    REQUIRE_ALIGNED(workspace);
    REQUIRE(static_cast<long long>(T) * k <= 0x7fffffffLL, INVMOE_ERR_UNSUPPORTED_SHAPE, "T * k exceeds 2^31 - 1");
  }
  if (T == 0) {
    if (plan == nullptr) return INVMOE_OK;
    return check_cuda(cudaMemsetAsync(plan, 0, (2 * static_cast<size_t>(E) + 1) * sizeof(int32_t), st),
                      "cudaMemsetAsync");
  }
  REQUIRE_PTR(logits); REQUIRE_PTR(topk_idx); REQUIRE_PTR(topk_w);
  rc = select_launch(logits, bias, T, E, k, score == INVMOE_SCORE_SOFTMAX, n_group, topk_group, renormalize != 0, scale,
                     topk_idx, topk_w, st);
  if (rc || plan == nullptr) return rc;
  return dispatch_launch(topk_idx, T, E, k, 0, nullptr, plan, nullptr, reinterpret_cast<int32_t*>(scratch(workspace)),
                         st);
}

int moe_route_select_backward(const float* logits, const int32_t* topk_idx, const float* dw, int T, int E, int k,
                              int score, int renormalize, float scale, float* dlogits, void* dlogits_bf16,
                              void* stream) {
  const int rc = check_select(T, E, k, score, 1, 1);
  if (rc) return rc;
  REQUIRE(dlogits != nullptr || dlogits_bf16 != nullptr || T == 0, INVMOE_ERR_INVALID_ARG,
          "dlogits and dlogits_bf16 are both NULL");
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(logits); REQUIRE_PTR(topk_idx); REQUIRE_PTR(dw);
  return select_bwd_launch(logits, topk_idx, dw, T, E, k, score == INVMOE_SCORE_SOFTMAX, renormalize != 0, scale,
                           dlogits, dlogits_bf16, static_cast<cudaStream_t>(stream));
}

int moe_router_backward(const void* x, const void* w_router, const void* dlogits_bf16, const float* dxp,
                        const int32_t* plan, const float* dx_shared, int T, int H, int E, int k, float* dx,
                        float* dw_router, void* workspace, size_t ws_bytes, void* stream) {
  REQUIRE(T >= 0 && H > 0 && E > 0 && k > 0 && k <= E && k <= 32, INVMOE_ERR_INVALID_ARG, "bad sizes");
  REQUIRE(H % 64 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 64", H);
  REQUIRE(E % 8 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "E=%d is not a multiple of 8", E);
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= kStatusBytes, INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  REQUIRE_ALIGNED(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dw_router)
      return check_cuda(cudaMemsetAsync(dw_router, 0, static_cast<size_t>(E) * H * 4, st), "cudaMemsetAsync");
    return INVMOE_OK;
  }
  REQUIRE_PTR(x); REQUIRE_PTR(w_router); REQUIRE_PTR(dlogits_bf16); REQUIRE_PTR(dxp); REQUIRE_PTR(plan);
  REQUIRE_PTR(dx);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(w_router); REQUIRE_ALIGNED(dlogits_bf16); REQUIRE_ALIGNED(dxp);
  REQUIRE_ALIGNED(dx);
  if (dx_shared) REQUIRE_ALIGNED(dx_shared);
  if (dw_router) REQUIRE_ALIGNED(dw_router);
  return router_backward_run(dlogits_bf16, x, w_router, dxp, plan, dx_shared, T, H, E, k, dx, dw_router,
                             status_word(workspace), st);
}

int add_rms_norm(const void* x, int x_type, const void* residual, int residual_type, const void* weight, int T, int H,
                 float eps, void* residual_out, void* out, void* q, float* scale, float* rstd, void* stream) {
  int rc = check_type(x_type, "x_type");
  if (rc == INVMOE_OK && residual != nullptr) rc = check_type(residual_type, "residual_type");
  if (rc == INVMOE_OK) rc = check_width(H);
  if (rc) return rc;
  REQUIRE(T >= 0, INVMOE_ERR_INVALID_ARG, "need T >= 0");
  REQUIRE(eps >= 0.0f, INVMOE_ERR_INVALID_ARG, "need eps >= 0");
  REQUIRE((q == nullptr) == (scale == nullptr), INVMOE_ERR_INVALID_ARG, "q and scale go together");
  if (T == 0) return INVMOE_OK;
  REQUIRE(out != nullptr || q != nullptr, INVMOE_ERR_INVALID_ARG, "out and q are both NULL");
  REQUIRE((residual == nullptr) == (residual_out == nullptr), INVMOE_ERR_INVALID_ARG,
          "residual and residual_out go together");
  REQUIRE_PTR(x); REQUIRE_PTR(weight);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(weight); REQUIRE_ALIGNED(residual); REQUIRE_ALIGNED(residual_out);
  REQUIRE_ALIGNED(out); REQUIRE_ALIGNED(q);
  REQUIRE(same_or_apart(residual_out, residual, matrix_bytes(T, H, residual_type)), INVMOE_ERR_INVALID_ARG,
          "residual_out overlaps residual without being it");
  return norm_launch(x, x_type == INVMOE_F32, residual, residual != nullptr && residual_type == INVMOE_F32, weight, T,
                     H, eps, residual_out, out, q, scale, rstd, static_cast<cudaStream_t>(stream));
}

size_t rms_norm_backward_workspace_size(int T, int H) {
  if (T <= 0 || H <= 0) return kStatusBytes;
  const int rows = norm_bwd_rows(T, H);
  return kStatusBytes + align_up(static_cast<size_t>((T - 1) / rows + 1) * H * sizeof(float), 256);
}

int add_rms_norm_backward(const void* dy, int dy_type, const void* x, int x_type, const void* weight,
                          const float* rstd, const void* dres, int T, int H, void* dx, float* dweight, void* workspace,
                          size_t ws_bytes, void* stream) {
  int rc = check_type(dy_type, "dy_type");
  if (rc == INVMOE_OK) rc = check_type(x_type, "x_type");
  if (rc == INVMOE_OK) rc = check_width(H);
  if (rc) return rc;
  REQUIRE(T >= 0, INVMOE_ERR_INVALID_ARG, "need T >= 0");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dweight != nullptr) {
    REQUIRE_PTR(workspace);
    REQUIRE(ws_bytes >= rms_norm_backward_workspace_size(T, H), INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
    REQUIRE_ALIGNED(workspace); REQUIRE_ALIGNED(dweight);
  }
  if (T == 0) {
    if (dweight == nullptr) return INVMOE_OK;
    return check_cuda(cudaMemsetAsync(dweight, 0, static_cast<size_t>(H) * 4, st), "cudaMemsetAsync");
  }
  REQUIRE_PTR(dy); REQUIRE_PTR(x); REQUIRE_PTR(weight); REQUIRE_PTR(rstd); REQUIRE_PTR(dx);
  REQUIRE_ALIGNED(dy); REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(weight); REQUIRE_ALIGNED(dx); REQUIRE_ALIGNED(dres);
  REQUIRE(same_or_apart(dx, dres, matrix_bytes(T, H, x_type)), INVMOE_ERR_INVALID_ARG, "dx overlaps dres without being it");
  return norm_bwd_launch(dy, dy_type == INVMOE_F32, x, x_type == INVMOE_F32, weight, rstd, dres, T, H, dx, dweight,
                         dweight != nullptr ? reinterpret_cast<float*>(scratch(workspace)) : nullptr, st);
}

int fp8_quantize(const void* x, int x_type, int banks, int rows, int cols, int block_rows, void* q, float* scale,
                 void* stream) {
  int rc = check_type(x_type, "x_type");
  if (rc) return rc;
  REQUIRE(banks >= 0 && rows >= 0 && cols > 0, INVMOE_ERR_INVALID_ARG, "need banks, rows >= 0 and cols > 0");
  REQUIRE(cols % 16 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "cols=%d is not a multiple of 16", cols);
  REQUIRE(block_rows == 1 || block_rows == 128, INVMOE_ERR_INVALID_ARG, "block_rows must be 1 or 128");
  if (banks == 0 || rows == 0) return INVMOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(q); REQUIRE_PTR(scale);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(q);
  return quantize_launch(x, x_type == INVMOE_F32, banks, rows, cols, block_rows, q, scale,
                         static_cast<cudaStream_t>(stream));
}

int moe_permute_rows(const void* x, const int32_t* plan, int T, int H, int E, int k, void* xp, void* stream) {
  REQUIRE(T >= 0 && H > 0 && E > 0 && k > 0 && k <= E && k <= 32, INVMOE_ERR_INVALID_ARG, "bad sizes");
  REQUIRE(H % 8 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 8", H);
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(x); REQUIRE_PTR(plan); REQUIRE_PTR(xp);
  REQUIRE_ALIGNED(x); REQUIRE_ALIGNED(xp);
  return permute_launch(x, plan + 2 * E + 1 + static_cast<long long>(T) * k, T, k, H, xp,
                        static_cast<cudaStream_t>(stream));
}

int moe_permute_fp8(const void* q, const float* scale, const int32_t* plan, int T, int H, int E, int k, void* xp,
                    float* xp_scale, void* stream) {
  REQUIRE(T >= 0 && E > 0 && k > 0 && k <= E && k <= 32, INVMOE_ERR_INVALID_ARG, "bad sizes");
  const int rc = check_width(H);
  if (rc) return rc;
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(q); REQUIRE_PTR(scale); REQUIRE_PTR(plan); REQUIRE_PTR(xp); REQUIRE_PTR(xp_scale);
  REQUIRE_ALIGNED(q); REQUIRE_ALIGNED(xp);
  return permute_fp8_launch(q, scale, plan + 2 * E + 1 + static_cast<long long>(T) * k, T, k, H, xp, xp_scale,
                            static_cast<cudaStream_t>(stream));
}

int fp8_gemm(const void* a, const float* a_scale, const void* b, const float* b_scale, int M, int N, int K, void* out,
             int out_type, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_type(out_type, "out_type");
  if (rc) return rc;
  REQUIRE(M >= 0 && N > 0 && K > 0, INVMOE_ERR_INVALID_ARG, "need M >= 0, N, K > 0");
  REQUIRE(K % 16 == 0, INVMOE_ERR_UNSUPPORTED_SHAPE, "K=%d is not a multiple of 16", K);
  REQUIRE(N <= 0x7fffff00 && K <= 0x7fffff00, INVMOE_ERR_UNSUPPORTED_SHAPE, "N=%d or K=%d is too large", N, K);
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= kStatusBytes, INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (M == 0) return INVMOE_OK;
  REQUIRE_PTR(a); REQUIRE_PTR(a_scale); REQUIRE_PTR(b); REQUIRE_PTR(b_scale); REQUIRE_PTR(out);
  REQUIRE_ALIGNED(a); REQUIRE_ALIGNED(b); REQUIRE_ALIGNED(out); REQUIRE_ALIGNED(workspace);
  Fp8Call c{};
  c.name = "fp8_gemm";
  c.a = a; c.a_scale = a_scale; c.rows = M; c.w = b; c.w_scale = b_scale; c.K = K; c.N = N;
  c.out = out; c.out_kind = out_type == INVMOE_F32 ? FP8_OUT_F32 : FP8_OUT_BF16;
  c.status = status_word(workspace);
  return fp8_gemm_run(c, static_cast<cudaStream_t>(stream));
}

int moe_grouped_swiglu_fp8(const void* xp, const float* xp_scale, const int32_t* plan, const void* w13,
                           const float* w13_scale, int T, int H, int E, int k, int F, void* h, float* h_scale,
                           void* workspace, size_t ws_bytes, void* stream) {
  const int rc = check_grouped(T, H, E, k, F);
  if (rc) return rc;
  REQUIRE(plan != nullptr || (E == 1 && k == 1), INVMOE_ERR_INVALID_ARG, "plan is NULL: only for E = k = 1");
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= kStatusBytes, INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(xp); REQUIRE_PTR(xp_scale); REQUIRE_PTR(w13); REQUIRE_PTR(w13_scale); REQUIRE_PTR(h);
  REQUIRE_PTR(h_scale);
  REQUIRE_ALIGNED(xp); REQUIRE_ALIGNED(w13); REQUIRE_ALIGNED(h); REQUIRE_ALIGNED(workspace);
  Fp8Call c{};
  c.name = "fp8_gate_up";
  c.a = xp; c.a_scale = xp_scale; c.rows = T * k; c.w = w13; c.w_scale = w13_scale; c.K = H; c.N = F;
  c.G = plan != nullptr ? E : 0;
  c.counts = plan; c.offsets = plan != nullptr ? plan + E : nullptr;
  c.out = h; c.out_scale = h_scale; c.out_kind = FP8_OUT_SWIGLU;
  c.status = status_word(workspace);
  return fp8_gemm_run(c, static_cast<cudaStream_t>(stream));
}

int moe_grouped_down_fp8(const void* h, const float* h_scale, const int32_t* plan, const void* w2,
                         const float* w2_scale, int T, int H, int E, int k, int F, float* y, void* workspace,
                         size_t ws_bytes, void* stream) {
  const int rc = check_grouped(T, H, E, k, F);
  if (rc) return rc;
  REQUIRE(plan != nullptr || (E == 1 && k == 1), INVMOE_ERR_INVALID_ARG, "plan is NULL: only for E = k = 1");
  REQUIRE_PTR(workspace);
  REQUIRE(ws_bytes >= kStatusBytes, INVMOE_ERR_WORKSPACE_TOO_SMALL, "workspace too small");
  if (T == 0) return INVMOE_OK;
  REQUIRE_PTR(h); REQUIRE_PTR(h_scale); REQUIRE_PTR(w2); REQUIRE_PTR(w2_scale); REQUIRE_PTR(y);
  REQUIRE_ALIGNED(h); REQUIRE_ALIGNED(w2); REQUIRE_ALIGNED(y); REQUIRE_ALIGNED(workspace);
  Fp8Call c{};
  c.name = "fp8_down";
  c.a = h; c.a_scale = h_scale; c.rows = T * k; c.w = w2; c.w_scale = w2_scale; c.K = F; c.N = H;
  c.G = plan != nullptr ? E : 0;
  c.counts = plan; c.offsets = plan != nullptr ? plan + E : nullptr;
  c.out = y; c.out_kind = FP8_OUT_F32;
  c.status = status_word(workspace);
  return fp8_gemm_run(c, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
