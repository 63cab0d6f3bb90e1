// route_token.cuh -- the choice of one token's experts by one warp, shared by the routing kernels and the one-kernel layer.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace invmoe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// How a logit is read: of an earlier kernel (plainly, or through the read-only path), or of another block of this one.
struct LoadPlain {
  __device__ __forceinline__ float operator()(const float* p) const { return *p; }
};
struct LoadReadOnly {
  __device__ __forceinline__ float operator()(const float* p) const { return __ldg(p); }
};
struct LoadL2 {
  __device__ __forceinline__ float operator()(const float* p) const { return __ldcg(p); }
};

// Total order key: larger = ranks earlier.  NaN -> 0 (below every number,
// including -inf); -0.0 and +0.0 map to the same key (a tie).
__device__ __forceinline__ uint32_t topk_key(float v) {
  if (v != v) return 0u;
  uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float topk_key_value(uint32_t key) {
  if (key == 0u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// One warp per token.  Lane l holds experts l, l+32, ... (EPL of them).  Each of
// the k rounds takes the warp-wide maximum of the order keys still in play
// (redux.sync max), then the lowest expert index holding that key (redux.sync
// min): a larger logit wins, an exact tie goes to the lower expert index, and a
// NaN (key 0) is taken only after every number, lowest index first.  The gate
// softmax is taken over the k selected logits in rank order, in fp32.  Lane j < k
// returns the j-th ranked expert and its gate.  Every routing kernel calls
// this one function, so they take the same decisions and compute the same gate bits.
template <int EPL, typename LOAD>
__device__ __forceinline__ void topk_choose(const float* row, LOAD ld, int E, int k, int lane, int& my_e, float& my_v) {
  uint32_t key[EPL];
  uint32_t live = 0u;   // bit i: expert i*32 + lane exists and has not been taken yet
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 32 + lane;
    key[i] = (e < E) ? topk_key(ld(row + e)) : 0u;
    if (e < E) live |= 1u << i;
  }
  my_e = 0;
  my_v = 0.0f;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (((live >> i) & 1u) && key[i] > best) best = key[i];
    const uint32_t gbest = __reduce_max_sync(kFull, best);
    uint32_t cand = 0xffffffffu;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i)
      if (((live >> i) & 1u) && key[i] == gbest) cand = static_cast<uint32_t>(i * 32 + lane);
    const int e = static_cast<int>(__reduce_min_sync(kFull, cand));
    if ((e & 31) == lane) live &= ~(1u << (e >> 5));
    if (lane == j) {
      my_e = e;
      my_v = topk_key_value(gbest);
    }
  }
}

// Lane j < k's gate, of the j-th logit that topk_choose left it.
__device__ __forceinline__ float topk_gate(float my_v, int k, int lane) {
  // w_j = exp(v_j - v_0) / sum_{i<k} exp(v_i - v_0), the sum in rank order
  const float v0 = __shfl_sync(kFull, my_v, 0);
  const float ex = (lane < k) ? expf(my_v - v0) : 0.0f;
  float s = 0.0f;
  for (int j = 0; j < k; ++j) s = __fadd_rn(s, __shfl_sync(kFull, ex, j));
  return __fdiv_rn(ex, s);
}

template <int EPL, typename LOAD>
__device__ __forceinline__ void topk_token(const float* row, LOAD ld, int E, int k, int lane, int& out_e, float& out_w) {
  float v;
  topk_choose<EPL>(row, ld, E, k, lane, out_e, v);
  out_w = topk_gate(v, k, lane);
}

// Larger = ranks earlier; NaN -> 1 (below every number, whose keys start at 0x007fffff); 0 is left for "not there"; -0 and
// +0 tie.
__device__ __forceinline__ uint32_t select_key(float v) {
  if (v != v) return 1u;
  const uint32_t b = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float select_key_value(uint32_t key) {
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
    if (i * 32 + lane < E) best = max(best, select_key(l[i]));
  SoftmaxStats s;
  const float m = select_key_value(__reduce_max_sync(kFull, best));
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

// One warp's choice for one token: lane j < k returns the j-th ranked expert; st: the row's statistics (SOFTMAX).  GROUPS: sk is the warp's own
// shared memory, E words and one per 32.
template <int EPL, bool SOFTMAX, bool GROUPS, typename LOAD>
__device__ __forceinline__ void select_choose(const float* row, LOAD ld, const SelectParams& p, uint32_t* sk, int lane,
                                              int& my_e, SoftmaxStats& st) {
  float l[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = i * 32 + lane < p.E ? ld(row + i * 32 + lane) : -INFINITY;
  st = SoftmaxStats{0.0f, 1.0f};
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
      key[i] = select_key(c);
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
    const uint32_t gkey = pairs ? select_key(__fadd_rn(select_key_value(ga), select_key_value(gb))) : ga;
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
  my_e = 0;
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
}

// Lane j < k's weight of expert my_e, the j-th ranked.
template <bool SOFTMAX, typename LOAD>
__device__ __forceinline__ float select_weight(const float* row, LOAD ld, const SelectParams& p, int my_e, const SoftmaxStats& st,
                                               int lane) {
  float s = 0.0f;
  if (lane < p.k) {
    const float lj = ld(row + my_e);
    s = SOFTMAX ? softmax_score(lj, st) : sigmoid_f32(lj);
  }
  if (p.renorm) {
    float sum = 0.0f;
    for (int j = 0; j < p.k; ++j) sum = __fadd_rn(sum, __shfl_sync(kFull, s, j));
    s = sum == 0.0f ? 0.0f : __fdiv_rn(s, sum);
  }
  return __fmul_rn(s, p.scale);
}

template <int EPL, bool SOFTMAX, bool GROUPS, typename LOAD>
__device__ __forceinline__ void select_token(const float* row, LOAD ld, const SelectParams& p, uint32_t* sk, int lane,
                                             int& out_e, float& out_w) {
  SoftmaxStats st;
  select_choose<EPL, SOFTMAX, GROUPS>(row, ld, p, sk, lane, out_e, st);
  out_w = select_weight<SOFTMAX>(row, ld, p, out_e, st, lane);
}

}  // namespace

}  // namespace invmoe
