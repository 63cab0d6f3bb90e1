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

namespace invmoe {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 256;

// Larger = ranks earlier; NaN -> 1 (below every number, whose keys start at 0x007fffff); 0 is left for "not there"; -0 and
// +0 tie.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t key) {
  if (key <= 1u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// 1 / (1 + exp(-l)); the reciprocal is correctly rounded, so it is the division's bits for fewer instructions.
__device__ __forceinline__ float sigmoid_f32(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// Shift and denominator of the softmax over a row held as l[i] = logit of expert i * 32 + lane; KEEP: l[i] becomes
// exp(logit - shift).  A row of -inf alone has shift 0 and denominator 0; a row with a NaN or +inf has a NaN denominator.
struct SoftmaxStats {
  float shift, total;
};
template <int EPL, bool KEEP>
__device__ __forceinline__ SoftmaxStats softmax_stats(float (&l)[EPL], int E, int lane) {
  uint32_t best = 0u;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i * 32 + lane < E) best = max(best, order_key(l[i]));
  SoftmaxStats s;
  const float m = key_value(__reduce_max_sync(kFull, best));
  s.shift = m == -INFINITY ? 0.0f : m;
  // e = (hi + lo * 2^-21) * 2^-21 up to 2^-42: hi <= 2^21, lo < 2^21, at most 1024 experts: no overflow in 32 bits
  unsigned hi = 0u, lo = 0u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (i * 32 + lane < E) {
      const float e = expf(__fsub_rn(l[i], s.shift));
      if (KEEP) l[i] = e;
      if (e <= 1.0f) {
        const float t = __fmul_rn(e, 2097152.0f);
        const unsigned h = static_cast<unsigned>(t);
        hi += h;
        lo += static_cast<unsigned>(__fmul_rn(__fsub_rn(t, static_cast<float>(h)), 2097152.0f));
      } else {
        bad = true;
      }
    }
  }
  hi = __reduce_add_sync(kFull, hi);
  lo = __reduce_add_sync(kFull, lo);
  const unsigned long long sum = (static_cast<unsigned long long>(hi) << 21) + lo;
  s.total = __any_sync(kFull, bad) ? __uint_as_float(0x7fc00000u)
                                   : __fmul_rn(__ull2float_rn(sum), 2.2737367544323206e-13f);   // 2^-42
  return s;
}

// p = exp(l - shift) / total of an e = exp(l - shift); an empty row's scores are 0.
__device__ __forceinline__ float softmax_share(float e, const SoftmaxStats& s) {
  return s.total == 0.0f ? 0.0f : __fdiv_rn(e, s.total);
}
__device__ __forceinline__ float softmax_score(float l, const SoftmaxStats& s) {
  return softmax_share(expf(__fsub_rn(l, s.shift)), s);
}

struct SelectParams {
  const float* logits;
  const float* bias;
  int T, E, k, n_group, topk_group, renorm;
  float scale;
  int32_t* idx;
  float* w;
};

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
  const float* row = p.logits + t * p.E;
  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = i * 32 + lane < p.E ? __ldg(row + i * 32 + lane) : -INFINITY;
  SoftmaxStats st{0.0f, 1.0f};
  if (SOFTMAX) st = softmax_stats<EPL, false>(l, p.E, lane);
  uint32_t key[EPL];                          // 0: no such expert, or its group is not kept
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0u;
    if (e < p.E) {
      float c = l[i];
      // (a second exp, not one kept from the statistics: with 1024 experts those registers would spill)
      if (p.bias != nullptr) c = __fadd_rn(SOFTMAX ? softmax_score(c, st) : sigmoid_f32(c), __ldg(p.bias + e));
      key[i] = order_key(c);
    }
  }
  if (GROUPS) {
    const int per = p.E / p.n_group;
    const bool pairs = p.bias != nullptr && per > 1;
    uint32_t ga = 0u, gb = 0u;                // lane g: the two largest keys of group g
    if (per % 32 == 0) {
      // a group is c whole registers of the warp: its two largest keys by warp maxima
      const int c = per / 32;
      uint32_t a = 0u, b = 0u;
      int left = c, g = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        b = max(b, min(a, key[i]));
        a = max(a, key[i]);
        if (--left == 0 && g < p.n_group) {
          const uint32_t t1 = __reduce_max_sync(kFull, a);
          uint32_t t2 = 0u;
          if (pairs) {
            const int first = __ffs(__ballot_sync(kFull, a == t1)) - 1;
            t2 = __reduce_max_sync(kFull, lane == first ? b : a);
          }
          if (lane == g) {
            ga = t1;
            gb = t2;
          }
          ++g;
          left = c;
          a = b = 0u;
        }
      }
    } else {
      uint32_t* sk = sm_keys + warp * (p.E + p.E / 32 + 1);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (i * 32 + lane < p.E) sk[i * 33 + lane] = key[i];
      __syncwarp();
      if (lane < p.n_group) {
        for (int j = 0; j < per; ++j) {
          const int e = lane * per + j;
          const uint32_t v = sk[e + (e >> 5)];
          gb = max(gb, min(ga, v));
          ga = max(ga, v);
        }
      }
    }
    const uint32_t gkey = pairs ? order_key(__fadd_rn(key_value(ga), key_value(gb))) : ga;
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const uint32_t o = __shfl_sync(kFull, gkey, g);
      if (o > gkey || (o == gkey && g < lane)) ++rank;
    }
    const unsigned kept = __ballot_sync(kFull, lane < p.n_group && rank < p.topk_group);
    if (per % 32 == 0) {
      int left = per / 32, g = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (!((kept >> g) & 1u)) key[i] = 0u;
        if (--left == 0) {
          ++g;
          left = per / 32;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = i * 32 + lane;
        if (e < p.E && !((kept >> (e / per)) & 1u)) key[i] = 0u;
      }
    }
  }
  // k rounds: the warp's largest key, the lowest expert that has it.  A lane keeps its two largest keys at hand and looks
  // through its experts again only when it has lost both (with 8 choices over 32 lanes about once a token; the vote makes
  // that a branch of the warp).  What it has lost are the first of its keys in the order (largest, lowest expert), so a look
  // begins behind the last of them.
  uint32_t best = 0u, second = 0u;
  int best_i = 0, second_i = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (key[i] > best) {
      second = best;
      second_i = best_i;
      best = key[i];
      best_i = i;
    } else if (key[i] > second) {
      second = key[i];
      second_i = i;
    }
  }
  bool spare = true;                          // `second` is still there
  int my_e = 0;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t top = __reduce_max_sync(kFull, best);
    const int e = static_cast<int>(__reduce_min_sync(kFull, best == top ? static_cast<uint32_t>(best_i * 32 + lane) : kFull));
    if (lane == j) my_e = e;
    const bool mine = (e & 31) == lane;
    if (__any_sync(kFull, mine && !spare)) {
      if (mine) {
        const uint32_t lost = best;
        const int lost_i = best_i;
        best = second = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const uint32_t v = key[i] < lost || (key[i] == lost && i > lost_i) ? key[i] : 0u;
          if (v > best) {
            second = best;
            second_i = best_i;
            best = v;
            best_i = i;
          } else if (v > second) {
            second = v;
            second_i = i;
          }
        }
        spare = true;
      }
    } else if (mine) {
      best = second;
      best_i = second_i;
      spare = false;
    }
  }
  float s = 0.0f;
  if (lane < p.k) {
    const float lj = __ldg(row + my_e);
    s = SOFTMAX ? softmax_score(lj, st) : sigmoid_f32(lj);
  }
  if (p.renorm) {
    float sum = 0.0f;
    for (int j = 0; j < p.k; ++j) sum = __fadd_rn(sum, __shfl_sync(kFull, s, j));
    s = sum == 0.0f ? 0.0f : __fdiv_rn(s, sum);
  }
  if (lane < p.k) {
    p.idx[t * p.k + lane] = my_e;
    p.w[t * p.k + lane] = __fmul_rn(s, p.scale);
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
