// route_select.cu -- expert choice by scores: sigmoid or softmax, a balance bias, expert groups, top-k, renormalised
// weights; and the gradient of the weights with respect to the logits.
//
// One warp per token, lane l holding experts l, l + 32, ...  Everything that decides a choice is either exact or a
// single correctly defined fp32 value, so the chosen experts do not depend on any summation order:
//   * without a bias the choice is by logit (both scores increase with it), so no score is computed for the losers;
//   * with a bias the choice is by score + bias, one fp32 addition; a group's value is the sum of its two largest;
//   * the softmax denominator is summed in fixed point (steps of 2^-42, integers), exact whatever the order.
// What bounds it for many tokens is instruction issue, not the row it reads (65536 x 256 in 8 groups, top 4 and 8: 76 us,
// 0.9 TB/s): a sigmoid per expert (8 per lane), the groups' maxima (two warp reductions each) and the k rounds, of which
// the searches were half (looking through the lane's experts every time one is lost: 86 us).  8192 tokens take 14.5 us
// with groups, 10.6 without; 4096 x 128 softmax 9, where half is launch.  A warp per token, not a thread: the row comes in
// whole lines, and every reduction is one instruction.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "route_token.cuh"

namespace invmoe {

namespace {

constexpr int kSelThreads = 256;

// Blocks per SM that the registers must leave room for: up to E = 256 at most 32 registers a thread, so that a batch of
// 8192 tokens is resident at once (64 warps per SM); above, 64 (8192 x 1024: 51 us with the 83 to 111 the compiler would
// take, 38.5 with 64).
constexpr int select_blocks(int epl) { return epl <= 8 ? 8 : 4; }

template <int EPL, bool SOFTMAX, bool GROUPS>
__global__ void __launch_bounds__(kSelThreads, select_blocks(EPL)) select_kernel(const SelectParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t sm_keys[];      // GROUPS: per warp E choice keys, padded by one word per 32
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * (kSelThreads / 32) + warp;
  if (t >= p.T) return;
  int e;
  float w;
  select_token<EPL, SOFTMAX, GROUPS>(p.logits + t * p.E, LoadReadOnly{}, p, sm_keys + warp * (p.E + p.E / 32 + 1), lane, e, w);
  if (lane < p.k) {
    p.idx[t * p.k + lane] = e;
    p.w[t * p.k + lane] = w;
  }
}

// Gradient of the weights: with s_j the chosen scores, w_j = s_j / sum_i s_i (0 where the sum is 0), d_j = dw_j, times scale:
//   sigmoid, plain          dl_j = d_j s_j (1 - s_j), other experts 0
//   sigmoid, renormalised   dl_j = w_j (1 - s_j) sum_i w_i (d_j - d_i)
//   softmax, renormalised   dl_j = w_j sum_i w_i (d_j - d_i)
//   softmax, plain          dl_e = -p_e sum_i d_i p_i for the experts not chosen,
//                           dl_j = p_j (sum_i p_i (d_j - d_i) + d_j r),  r = the share of the experts not chosen
// In this form nothing cancels but what dw itself cancels: 1 - s_j is sigmoid(-l_j), and the sum over the chosen goes over
// differences instead of d_j less the mean, which of a confident expert (w_j or p_j near 1) leaves rounding errors alone.
// No quotient of a score but w_j either, so tiny scores do not overflow.
// One warp per token; an entry of topk_idx outside [0, E) takes no part.  Bound by writing the row, which is written as if
// nothing were chosen and then corrected at the k chosen entries (8192 x 1024, renormalised sigmoid: 8.6 us for 34 MB, half
// as much again when every column was compared with every choice; 8192 x 256: 5.4 us); the plain softmax by its exponentials
// and divisions (8192 x 1024: 28 us, of which the sum over the experts not chosen is 2).
template <int EPL, bool SOFTMAX>
__global__ void __launch_bounds__(kSelThreads, EPL <= 8 ? 5 : 4)
    select_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, const float* __restrict__ dw,
                      int T, int E, int k, int renorm, float scale, float* __restrict__ dl,
                      __nv_bfloat16* __restrict__ dl_bf16) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * (kSelThreads / 32) + (threadIdx.x >> 5);
  if (t >= T) return;
  const float* row = logits + t * E;
  // only a softmax that is not renormalised has a gradient for the experts not chosen, and needs every score in it
  const bool dense = SOFTMAX && !renorm;
  SoftmaxStats st{0.0f, 1.0f};
  float l[SOFTMAX ? EPL : 1];
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = i * 32 + lane < E ? __ldg(row + i * 32 + lane) : -INFINITY;
    st = softmax_stats<EPL, true>(l, E, lane);
  }
  int e = -1;
  float s = 0.0f, d = 0.0f, comp = 1.0f;         // comp: ds / dl = s * comp
  if (lane < k) {
    e = __ldg(idx + t * k + lane);
    if (e < 0 || e >= E) e = -1;
    if (e >= 0) {
      const float lj = __ldg(row + e);
      s = SOFTMAX ? softmax_score(lj, st) : sigmoid_f32(lj);
      if (!SOFTMAX) comp = sigmoid_f32(-lj);
      d = __ldg(dw + t * k + lane);
    }
  }
  float v = 0.0f, all = 0.0f;                    // of the chosen expert's entry, and of every other one's, before scale
  if (renorm) {
    float sum = 0.0f;
    for (int j = 0; j < k; ++j) sum += __shfl_sync(kFull, s, j);
    const float w = sum == 0.0f ? 0.0f : __fdiv_rn(s, sum);
    float acc = 0.0f;
    for (int j = 0; j < k; ++j)
      acc = fmaf(__shfl_sync(kFull, w, j), __fsub_rn(d, __shfl_sync(kFull, d, j)), acc);
    v = w * comp * acc;
  } else {
    v = d * s * comp;
  }
  if constexpr (SOFTMAX) {
    if (dense) {
      // D: the sum of the slots that chose the expert; `first`: the first of them, which stands for it below
      float D = 0.0f, rest = 0.0f;
      bool first = e >= 0;
      unsigned mine = 0u;                        // bit i: expert i * 32 + lane is chosen
      for (int j = 0; j < k; ++j) {
        const int ej = __shfl_sync(kFull, e, j);
        const float dj = __shfl_sync(kFull, d, j);
        all = fmaf(dj, __shfl_sync(kFull, s, j), all);
        if (ej == e) {
          D += dj;
          if (j < lane) first = false;
        }
        if (ej >= 0 && (ej & 31) == lane) mine |= 1u << (ej >> 5);
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i * 32 + lane < E && !((mine >> i) & 1u)) rest += l[i];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) rest += __shfl_xor_sync(kFull, rest, o);
      const float once = first ? s : 0.0f;
      float acc = __fmul_rn(D, softmax_share(rest, st));
      for (int j = 0; j < k; ++j)
        acc = fmaf(__shfl_sync(kFull, once, j), __fsub_rn(D, __shfl_sync(kFull, D, j)), acc);
      v = s * acc;
    }
  }
  if (!dense) {
    // an expert chosen twice gets both
    float both = 0.0f;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(kFull, e, j);
      const float vj = __shfl_sync(kFull, v, j);
      if (ej == e) both += vj;
    }
    v = both;
  }
  v = __fmul_rn(v, scale);
  all = __fmul_rn(all, scale);
  // the row as if nothing were chosen, then the chosen entries: the warp's stores to one address are in this order
  float* out = dl != nullptr ? dl + t * E : nullptr;
  __nv_bfloat16* out_bf16 = dl_bf16 != nullptr ? dl_bf16 + t * E : nullptr;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int c = i * 32 + lane;
    if (c < E) {
      float g = 0.0f;
      if constexpr (SOFTMAX)
        if (dense) g = __fsub_rn(0.0f, __fmul_rn(all, softmax_share(l[i], st)));
      if (out != nullptr) out[c] = g;
      if (out_bf16 != nullptr) out_bf16[c] = __float2bfloat16_rn(g);
    }
  }
  __syncwarp();
  if (e >= 0) {
    if (out != nullptr) out[e] = v;
    if (out_bf16 != nullptr) out_bf16[e] = __float2bfloat16_rn(v);
  }
}

template <int EPL>
cudaError_t select_epl(const SelectParams& p, int softmax, dim3 g, cudaStream_t st) {
  const dim3 b(kSelThreads);
  if (p.n_group > 1) {
    const size_t smem = p.E / p.n_group % 32 == 0 ? 0 : (kSelThreads / 32) * (static_cast<size_t>(p.E) + p.E / 32 + 1) * 4;
    return softmax ? launch_kernel(select_kernel<EPL, true, true>, g, b, smem, st, p)
                   : launch_kernel(select_kernel<EPL, false, true>, g, b, smem, st, p);
  }
  return softmax ? launch_kernel(select_kernel<EPL, true, false>, g, b, 0, st, p)
                 : launch_kernel(select_kernel<EPL, false, false>, g, b, 0, st, p);
}

template <int EPL>
cudaError_t select_bwd_epl(const float* logits, const int32_t* idx, const float* dw, int T, int E, int k, int softmax,
                           int renorm, float scale, float* dl, void* dl_bf16, dim3 g, cudaStream_t st) {
  __nv_bfloat16* db = static_cast<__nv_bfloat16*>(dl_bf16);
  return softmax ? launch_kernel(select_bwd_kernel<EPL, true>, g, dim3(kSelThreads), 0, st, logits, idx, dw, T, E, k,
                                 renorm, scale, dl, db)
                 : launch_kernel(select_bwd_kernel<EPL, false>, g, dim3(kSelThreads), 0, st, logits, idx, dw, T, E, k,
                                 renorm, scale, dl, db);
}

dim3 warp_per_token(int T) {
  return dim3(static_cast<unsigned>((static_cast<long long>(T) * 32 + kSelThreads - 1) / kSelThreads));
}

}  // namespace

int select_launch(const float* logits, const float* bias, int T, int E, int k, int softmax, int n_group, int topk_group,
                  int renorm, float scale, int32_t* idx, float* w, cudaStream_t st) {
  // all groups kept: the choice is over every expert, no group value matters
  const SelectParams p{logits, bias, T, E, k, topk_group == n_group ? 1 : n_group, topk_group, renorm, scale, idx, w};
  const dim3 g = warp_per_token(T);
  const int epl = (E + 31) / 32;
  ProfScope prof("route_select", st);
  cudaError_t e;
  if (epl <= 1) e = select_epl<1>(p, softmax, g, st);
  else if (epl <= 2) e = select_epl<2>(p, softmax, g, st);
  else if (epl <= 4) e = select_epl<4>(p, softmax, g, st);
  else if (epl <= 8) e = select_epl<8>(p, softmax, g, st);
  else if (epl <= 16) e = select_epl<16>(p, softmax, g, st);
  else e = select_epl<32>(p, softmax, g, st);
  return check_cuda(e, "select_kernel");
}

int select_bwd_launch(const float* logits, const int32_t* idx, const float* dw, int T, int E, int k, int softmax,
                      int renorm, float scale, float* dl, void* dl_bf16, cudaStream_t st) {
  const dim3 g = warp_per_token(T);
  const int epl = (E + 31) / 32;
  ProfScope prof("route_select_bwd", st);
  cudaError_t e;
  if (epl <= 1) e = select_bwd_epl<1>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  else if (epl <= 2) e = select_bwd_epl<2>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  else if (epl <= 4) e = select_bwd_epl<4>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  else if (epl <= 8) e = select_bwd_epl<8>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  else if (epl <= 16) e = select_bwd_epl<16>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  else e = select_bwd_epl<32>(logits, idx, dw, T, E, k, softmax, renorm, scale, dl, dl_bf16, g, st);
  return check_cuda(e, "select_bwd_kernel");
}

}  // namespace invmoe
