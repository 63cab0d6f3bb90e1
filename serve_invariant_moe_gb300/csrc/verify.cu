// verify.cu -- drafted tokens checked against the target's probabilities, from given random numbers.
//
// With p_i = softmax(z_i / tau) of a request's target rows and q_i of its draft rows, draft token x_i is accepted while
// u_i q_i(x_i) < p_i(x_i).  The token after the n accepted ones is drawn by a race of exponential noise e: the largest
// w_j / e_j, where w = max(p_n - q_n, 0) after a rejection and p_n otherwise, which draws j with probability w_j / sum w.  So
// every emitted token has the target's distribution, and which one it is follows from the logits and the given numbers alone.
//
// Two kernels: the statistics (maximum, sum of exponentials) of every row that counts, a block per chunk of kChunk logits;
// then acceptance and the race on the one row that is left, by as many blocks of a request as are resident, the last one to
// finish joining them.  Bound by reading the logits once and, for the row that is drawn from, once more, with the noise.
// The chunks and the order in which they are joined follow from V alone, and the largest score is the same however the race
// is shared out, so a request's bits do not depend on the batch.
// 64 requests of at most 4 drafts, 151552 tokens, fp32: 48 us (99 at first: expf and its special cases kept the
// statistics at 56 us, and a racing block per chunk, each with the whole decision to take, the choice at 50).  With all four
// drafts the statistics read 349 MB at 6.7 TB/s; the choice is bound by latency, 3.3 TB/s: each of its blocks takes the
// decision (chunks, draft tokens and their logits, one load behind the other) before it knows which row to read.  One request:
// 9 us, two launches and that chain.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace invmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;                          // logits of a thread of the statistics
constexpr int kChunk = kThreads * kPer;
constexpr int kRacePer = 16;                      // of the race, which holds two rows and the noise
constexpr int kRaceChunk = kThreads * kRacePer;

// NaN counts as no logit at all; +inf as the largest finite number, so that it takes all the mass.
__device__ __forceinline__ float usable(float z) { return fminf(fmaxf(z, -INFINITY), FLT_MAX); }

struct Scale {
  bool greedy;
  float inv;                                      // 1 / tau; 1 for a greedy request
  float inv2;                                     // log2(e) / tau
};
__device__ __forceinline__ Scale scale_of(const VerifyCall& p, int b) {
  const float tau = p.temperature != nullptr ? __ldg(p.temperature + b) : p.tau;
  const bool greedy = !(tau > 0.0f);
  // (not 0 for an infinite temperature either: -inf times it has to stay -inf)
  const float inv = greedy ? 1.0f : fminf(fmaxf(__frcp_rn(tau), FLT_MIN), FLT_MAX);
  return {greedy, inv, fminf(__fmul_rn(inv, 1.4426950408889634f), FLT_MAX)};
}

// 2^x within 2^-22, 0 below the normal numbers.  A weight is one subtraction, one product and one of these: with expf and
// its cases the statistics kernel was bound by instructions.  Its argument has been rounded three times (the difference,
// log2(e) / tau, their product), 3 x 2^-24 of it: at most 2e-5 of a weight, at the argument of -104 nats where nothing is left.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// exp((z - m) / tau) for a finite m; 0 for a logit of -inf.
__device__ __forceinline__ float weight(float z, float m, float inv2) {
  return exp2_approx(__fmul_rn(__fsub_rn(z, m), inv2));
}
// What to subtract from a chunk's logits: its maximum, or 0 where it has none.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ int drafts_of(const VerifyCall& p, int b) {
  return p.n_draft != nullptr ? max(0, min(p.D, __ldg(p.n_draft + b))) : p.D;
}

// Place of the i-th of a thread's logits in its chunk: vectors of 8 or, where rows do not start on 16 bytes, single ones.
template <bool VEC>
__device__ __forceinline__ int place(int i) {
  return VEC ? ((i >> 3) * kThreads + static_cast<int>(threadIdx.x)) * 8 + (i & 7)
             : i * kThreads + static_cast<int>(threadIdx.x);
}

// This thread's elements of a row from `first` on; `fill` behind the row's end.
template <typename T, bool VEC, int PER>
__device__ __forceinline__ void load_chunk(const T* row, int first, int V, float fill, float (&z)[PER]) {
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < PER / 8; ++v) {
      const int c = first + (v * kThreads + static_cast<int>(threadIdx.x)) * 8;
      float t[8];
      if (c + 8 <= V) {
        load8(row + c, t);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = c + i < V ? static_cast<float>(row[c + i]) : fill;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) z[v * 8 + i] = t[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = first + i * kThreads + static_cast<int>(threadIdx.x);
      z[i] = c < V ? static_cast<float>(row[c]) : fill;
    }
  }
}

struct Stats {
  float max, sum;
  int arg, pad;                                   // lowest index of the maximum (greedy requests)
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) verify_stats_kernel(const VerifyCall p) {
  // in this order: the next kernel reads the call's inputs as soon as every block has triggered, and whoever wrote them has
  // completed only behind the wait
  pdl_wait();
  pdl_trigger();
  __shared__ Stats s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = static_cast<int>(blockIdx.x % p.chunks);
  const long long row = blockIdx.x / p.chunks;    // a request's target rows, then its draft rows
  const int b = static_cast<int>(row / p.rows), i = static_cast<int>(row - static_cast<long long>(b) * p.rows);
  if (chunk == 0 && i == 0 && threadIdx.x == 0) p.done[b] = 0;
  const int n = drafts_of(p, b);
  const Scale sc = scale_of(p, b);
  const bool target = i <= p.D;
  if (target ? i > n : i - (p.D + 1) >= n || sc.greedy) return;
  const T* z_row = target ? static_cast<const T*>(p.logits) + (static_cast<long long>(b) * (p.D + 1) + i) * p.V
                          : static_cast<const T*>(p.draft_logits) + (static_cast<long long>(b) * p.D + i - (p.D + 1)) * p.V;
  float z[kPer];
  load_chunk<T, VEC>(z_row, chunk * kChunk, p.V, -INFINITY, z);
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    z[j] = usable(z[j]);
    m = fmaxf(m, z[j]);
  }
  // a warp's own maximum and sum first, so that the block meets once
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
  const float shift = shift_of(m);
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) s += weight(z[j], shift, sc.inv2);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
  int arg = 0x7fffffff;
  if (sc.greedy) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (z[j] == m) arg = min(arg, place<VEC>(j));
    arg = __reduce_min_sync(kFull, arg);
  }
  if (lane == 0) s_warp[warp] = Stats{m, s, arg, 0};
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = fmaxf(m, s_warp[w].max);
  s = 0.0f;
  arg = 0x7fffffff;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    s += s_warp[w].sum * weight(s_warp[w].max, shift_of(m), sc.inv2);
    if (s_warp[w].max == m) arg = min(arg, s_warp[w].arg);
  }
  static_cast<Stats*>(p.stats)[row * p.chunks + chunk] = Stats{m, s, chunk * kChunk + arg, 0};
}

// A row's statistics from its chunks': lane l joins chunks l, l + 32, ... ascending, then a xor butterfly.  `first`: the
// lane's first chunk, loaded by the caller.
__device__ __forceinline__ Stats join(const Stats& first, const Stats* part, int chunks, float inv2, int lane) {
  float m = first.max;
  for (int c = lane + 32; c < chunks; c += 32) m = fmaxf(m, part[c].max);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
  const float shift = shift_of(m);
  float s = first.sum * weight(first.max, shift, inv2);
  int arg = first.max == m ? first.arg : 0x7fffffff;
  for (int c = lane + 32; c < chunks; c += 32) {
    const Stats t = part[c];
    s += t.sum * weight(t.max, shift, inv2);
    if (t.max == m) arg = min(arg, t.arg);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
  return Stats{m, s, static_cast<int>(__reduce_min_sync(kFull, arg)), 0};
}

// A thread's best racer so far, its places ascending: the larger w / e wins, then the lower place.
struct Racer {
  float score = -1.0f;
  int at = 0;
  __device__ __forceinline__ void take(float w, float e_inv, int j) {
    const float v = __fmul_rn(w, e_inv);
    if (w > 0.0f && v > score && v >= 0.0f) {      // (a noise that is negative, -0 or NaN takes no part)
      score = v;
      at = j;
    }
  }
  // Comparable over threads; 0 is nobody.
  __device__ __forceinline__ unsigned long long key() const {
    if (score < 0.0f) return 0ull;
    return (static_cast<unsigned long long>(__float_as_uint(score)) << 32) | (0xffffffffu - static_cast<unsigned>(at));
  }
};
__device__ __forceinline__ unsigned long long warp_best(unsigned long long v) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v = max(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_choose_kernel(const VerifyCall p) {
  __shared__ Stats s_row[2 * kVerifyMaxDrafts + 1];
  __shared__ float s_z[2 * kVerifyMaxDrafts + 1];  // the row's logit of its draft token
  __shared__ int s_x[kVerifyMaxDrafts];
  __shared__ unsigned long long s_best[kThreads / 32];
  __shared__ int s_n, s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = static_cast<int>(blockIdx.x / p.racing), first_chunk = static_cast<int>(blockIdx.x % p.racing);
  const int D = p.D, V = p.V;
  const int n_draft = drafts_of(p, b);
  const Scale sc = scale_of(p, b);
  // what needs no decision is on its way first: the noise, and behind the statistics' kernel every row's chunks, the draft
  // tokens and their logits.  (Inputs may be read before that kernel ends: this one begins when all of its blocks are past
  // their wait for what came before.  64 requests 50.6 -> 47.9 us, one 9.5 -> 9.0.)
  float e[kRacePer];
  if (!sc.greedy) load_chunk<float, VEC>(p.noise + static_cast<long long>(b) * V, first_chunk * kRaceChunk, V, 1.0f, e);
  pdl_wait();
  pdl_trigger();
  if (sc.greedy && first_chunk != 0) return;            // nothing to draw: one block reads the maxima
  const Stats* part = static_cast<const Stats*>(p.stats) + static_cast<long long>(b) * p.rows * p.chunks;
  const T* logits = static_cast<const T*>(p.logits) + static_cast<long long>(b) * (D + 1) * V;
  const T* drafts = static_cast<const T*>(p.draft_logits) + static_cast<long long>(b) * D * V;
  const bool has_q = p.draft_logits != nullptr;
  for (int r0 = warp; r0 < p.rows; r0 += 2 * (kThreads / 32)) {
    Stats first[2];
    int x[2];
    float z[2];
    bool counts[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + h * (kThreads / 32), i = r <= D ? r : r - (D + 1);
      counts[h] = r < p.rows && (r <= D ? r <= n_draft : i < n_draft && !sc.greedy);
      first[h] = Stats{-INFINITY, 0.0f, 0x7fffffff, 0};
      if (counts[h] && lane < p.chunks) first[h] = part[static_cast<long long>(r) * p.chunks + lane];
      x[h] = counts[h] && i < n_draft ? __ldg(p.draft_tokens + static_cast<long long>(b) * D + i) : -1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + h * (kThreads / 32), i = r <= D ? r : r - (D + 1);
      z[h] = -INFINITY;
      if (x[h] >= 0 && x[h] < V) z[h] = static_cast<float>((r <= D ? logits : drafts)[static_cast<long long>(i) * V + x[h]]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + h * (kThreads / 32);
      if (!counts[h]) continue;
      const Stats t = join(first[h], part + static_cast<long long>(r) * p.chunks, p.chunks, sc.inv2, lane);
      if (lane == 0) {
        s_row[r] = t;
        s_z[r] = usable(z[h]);
        if (r < n_draft) s_x[r] = x[h];
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    bool ok = false;
    if (lane < n_draft) {
      const int x = s_x[lane];
      const Stats t = s_row[lane];
      if (x >= 0 && x < V && t.max > -INFINITY) {
        if (sc.greedy) {
          ok = x == t.arg;
        } else {
          // u q < p over the common denominators: u e_q S_p < e_p S_q
          const float ep = weight(s_z[lane], t.max, sc.inv2);
          float eq = 1.0f, sq = 1.0f;
          if (has_q) {
            const Stats d = s_row[D + 1 + lane];
            eq = d.max > -INFINITY ? weight(s_z[D + 1 + lane], d.max, sc.inv2) : 0.0f;
            sq = d.max > -INFINITY ? d.sum : 1.0f;
          }
          const float u = __ldg(p.accept_u + static_cast<long long>(b) * D + lane);
          ok = static_cast<double>(u) * eq * t.sum < static_cast<double>(ep) * sq;
        }
      }
    }
    const unsigned no = ~__ballot_sync(kFull, ok);
    if (lane == 0) s_n = no == 0u ? 32 : __ffs(no) - 1;
  }
  __syncthreads();
  const int n = s_n;                              // accepted; row n gives the next token
  const Stats t = s_row[n];
  const bool rejected = n < n_draft;
  const T* z_row = logits + static_cast<long long>(n) * V;
  const T* q_row = drafts + static_cast<long long>(n) * V;
  const float* noise = p.noise + static_cast<long long>(b) * V;
  const float inv_p = __frcp_rn(t.sum);
  const int race_chunks = (V - 1) / kRaceChunk + 1;
  Racer best;
  if (!sc.greedy && t.max > -INFINITY) {
    const Stats d = rejected && has_q ? s_row[D + 1 + n] : Stats{-INFINITY, 0.0f, 0, 0};
    const bool some_q = d.max > -INFINITY;
    const float inv_q = some_q ? __frcp_rn(d.sum) : 0.0f;
    const int x = rejected && !has_q ? s_x[n] : -1;              // what a drafter without probabilities drew
    for (int chunk = first_chunk; chunk < race_chunks; chunk += p.racing) {
      float z[kRacePer];
      if (chunk != first_chunk) load_chunk<float, VEC>(noise, chunk * kRaceChunk, V, 1.0f, e);
      load_chunk<T, VEC>(z_row, chunk * kRaceChunk, V, -INFINITY, z);
      if (some_q) {
        float q[kRacePer];
        load_chunk<T, VEC>(q_row, chunk * kRaceChunk, V, -INFINITY, q);
#pragma unroll
        for (int j = 0; j < kRacePer; ++j) {
          const float pj = __fmul_rn(weight(usable(z[j]), t.max, sc.inv2), inv_p);
          const float qj = __fmul_rn(weight(usable(q[j]), d.max, sc.inv2), inv_q);
          best.take(__fsub_rn(pj, qj), rcp_approx(e[j]), chunk * kRaceChunk + place<VEC>(j));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kRacePer; ++j) {
          const int at = chunk * kRaceChunk + place<VEC>(j);
          const float pj = __fmul_rn(weight(usable(z[j]), t.max, sc.inv2), inv_p);
          if (at != x) best.take(pj, rcp_approx(e[j]), at);
        }
      }
    }
  }
  // the block's best in thread 0
  auto block_best = [&](const Racer& r) {
    unsigned long long v = warp_best(r.key());
    if (lane == 0) s_best[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v = max(v, s_best[w]);
    return v;
  };
  unsigned long long first = block_best(best);
  unsigned long long* racers = static_cast<unsigned long long*>(p.racers) + static_cast<long long>(b) * p.racing;
  if (threadIdx.x == 0) {
    s_last = 1;
    if (!sc.greedy && p.racing > 1) {
      racers[first_chunk] = first;
      __threadfence();
      s_last = atomicAdd(p.done + b, 1) == p.racing - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  int token = t.max > -INFINITY ? t.arg : -1;
  if (!sc.greedy) {
    if (p.racing > 1) {                           // every warp for itself
      first = 0ull;
      for (int c = lane; c < p.racing; c += 32) first = max(first, __ldcg(racers + c));
      first = warp_best(first);
    }
    if (first == 0ull && rejected && t.max > -INFINITY) {
      // p - q is nowhere above 0 (they are equal, and the draft token was none of the vocabulary's): this block draws from p
      Racer alone;
      for (int c = threadIdx.x; c < V; c += kThreads)
        alone.take(__fmul_rn(weight(usable(static_cast<float>(z_row[c])), t.max, sc.inv2), inv_p), rcp_approx(noise[c]), c);
      first = block_best(alone);
    }
    token = first == 0ull ? -1 : static_cast<int>(0xffffffffu - static_cast<unsigned>(first));
  }
  if (warp != 0) return;
  if (lane == 0) p.n_accepted[b] = n;
  for (int i = lane; i <= D; i += 32) {
    int x = -1;
    float lp = 0.0f;
    if (i <= n) {
      x = i < n ? s_x[i] : token;
      const Stats r = s_row[i];
      const float z = i < n ? s_z[i] : x < 0 ? 0.0f : usable(static_cast<float>(logits[static_cast<long long>(i) * V + x]));
      lp = x < 0 ? -INFINITY : __fsub_rn(__fmul_rn(__fsub_rn(z, r.max), sc.inv), logf(r.sum));
    }
    p.tokens[static_cast<long long>(b) * (D + 1) + i] = x;
    p.logp[static_cast<long long>(b) * (D + 1) + i] = lp;
  }
}

}  // namespace

int verify_chunks(int V) { return (V - 1) / kChunk + 1; }
int verify_race_chunks(int V) { return (V - 1) / kRaceChunk + 1; }

int verify_launch(VerifyCall c, bool f32, cudaStream_t st) {
  const bool vec = c.V % (f32 ? 4 : 8) == 0;
  int sms = 0;
  const int rc = device_sm_count(&sms);
  if (rc) return rc;
  // Every racing block decides for itself, so no more of them than are resident, four to a multiprocessor (64 requests with
  // 1216 blocks of one chunk took 33 us for this kernel, 27 with two blocks to a multiprocessor, 25 with four of half the
  // chunk).  The largest score is the same however the chunks are shared out.
  const int race_chunks = verify_race_chunks(c.V), resident = 4 * sms / c.B;
  c.racing = resident < 1 ? 1 : resident < race_chunks ? resident : race_chunks;
  const dim3 g1(static_cast<unsigned>(static_cast<long long>(c.B) * c.rows * c.chunks)), g2(c.B * c.racing);
  {
    ProfScope prof("verify_stats", st);
    const cudaError_t e =
        f32 ? vec ? launch_kernel(verify_stats_kernel<float, true>, g1, dim3(kThreads), 0, st, c)
                  : launch_kernel(verify_stats_kernel<float, false>, g1, dim3(kThreads), 0, st, c)
        : vec ? launch_kernel(verify_stats_kernel<__nv_bfloat16, true>, g1, dim3(kThreads), 0, st, c)
              : launch_kernel(verify_stats_kernel<__nv_bfloat16, false>, g1, dim3(kThreads), 0, st, c);
    const int rc = check_cuda(e, "verify_stats_kernel");
    if (rc) return rc;
  }
  ProfScope prof("verify_choose", st);
  const cudaError_t e =
      f32 ? vec ? launch_kernel(verify_choose_kernel<float, true>, g2, dim3(kThreads), 0, st, c)
                : launch_kernel(verify_choose_kernel<float, false>, g2, dim3(kThreads), 0, st, c)
      : vec ? launch_kernel(verify_choose_kernel<__nv_bfloat16, true>, g2, dim3(kThreads), 0, st, c)
            : launch_kernel(verify_choose_kernel<__nv_bfloat16, false>, g2, dim3(kThreads), 0, st, c);
  return check_cuda(e, "verify_choose_kernel");
}

}  // namespace invmoe
