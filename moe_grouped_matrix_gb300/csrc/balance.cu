// The losses that keep a router's experts evenly loaded, with the experts' loads,
// and the gradient of the losses with respect to the logits.
//
//   p[t]   softmax of token t's logits, or their sigmoids over the sum of these
//   f[s]   shares of sequence s's slots that each expert got (no gradient)
//   balance = E/N sum_t <f[s(t)], p[t]>        z = 1/N sum_t lse(l[t])^2
//   dl = d0 E/N p (f - <f, p>) + d1 2/N lse softmax(l)
// and with sigmoid scores the first term times 1 - sigmoid(l).  f is known only when all
// tokens have been counted, but sum_t <f, p[t]> = <f, sum_t p[t]>: one pass over the
// logits sums p by expert.
//
// Forward: a warp takes a token, its lanes the experts, sums in registers; the CTAs of a
// cluster take runs of one sequence's tokens and join their sums through shared memory,
// each those of a slice of the experts.  Up to 2048 tokens of one sequence are one cluster
// of up to 16 CTAs, which ends with the losses; more clusters leave their sums to a second
// kernel, again one cluster.  All joins have a fixed order.
//
// Bound by latency: 192 tokens, 2 of 8 experts 4.8 us and the gradient 2.1; 4096 tokens, 8
// of 128 experts 9.8 us (the first kernel 6.4, of which 2 to 4 are the tokens, the join 3)
// and 3.1 for 1 MB of logits.  Of many logits by instructions: 16384 tokens of 250 f32 logits
// in 16 sequences, sigmoid scores, 15 us and 9.9 for 16 MB (2.4 and 4.8 at memory's rate), of
// which 5.9 and 6.6 are issue slots: 420 and 467 instructions a token.
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWarps = 16, kBackWarps = 8;
// CTAs that a forward pass is cut into, about: two for each SM of a GB300.  A constant, as the size of the scratch,
// which is asked for without a device, follows from it.
constexpr int kCtas = 304;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // NaN does not count
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// How a row of experts lies in a warp: V values a lane, in units of UE consecutive ones (whole 16-byte
// loads where the rows allow them, else single values).
template <int V, class T>
constexpr int kUnit = V < 16 / int(sizeof(T)) ? V : 16 / int(sizeof(T));
template <int UE>
__device__ __forceinline__ int expert_of(int i) {
  return (i / UE * 32 + int(threadIdx.x & 31)) * UE + i % UE;
}

// The lane's logits (past the last expert: -inf).  UE > 1: experts is a multiple of it, the row aligned to it.
template <int V, int UE, class T>
__device__ __forceinline__ void load_row(const T* row, int experts, float (&l)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += UE) {
    const int e = expert_of<UE>(i);
    if (e < experts) {
      using Bits = std::conditional_t<sizeof(T) * UE == 16, uint4, std::conditional_t<sizeof(T) * UE == 8, uint2,
                   std::conditional_t<sizeof(T) * UE == 4, uint32_t, uint16_t>>>;
      const Bits bits = __ldg(reinterpret_cast<const Bits*>(row + e));
      const T* t = reinterpret_cast<const T*>(&bits);
#pragma unroll
      for (int j = 0; j < UE; ++j) l[i + j] = as_float(t[j]);
    } else {
#pragma unroll
      for (int j = 0; j < UE; ++j) l[i + j] = -INFINITY;
    }
  }
}

template <int V>
__device__ __forceinline__ float row_max(const float (&l)[V]) {
  float high = l[0];
#pragma unroll
  for (int i = 1; i < V; ++i) high = fmaxf(high, l[i]);
  return warp_max(high);
}
// Whether a row has anything but -inf, high its largest (NaN counts as something).
template <int V>
__device__ __forceinline__ bool any_logit(const float (&l)[V], float high) {
  if (high != -INFINITY) return true;
  bool some = false;
#pragma unroll
  for (int i = 0; i < V; ++i) some |= l[i] != -INFINITY;
  return __any_sync(0xffffffffu, some);
}
// l becomes exp(l - high); returns the sum over the row.
template <int V>
__device__ __forceinline__ float exponentials(float (&l)[V], float high) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += l[i] = expf(l[i] - high);
  return warp_sum(sum);
}

// The sigmoids of a row up to a common factor, from its logits l and ex = exp(l - high), and what 1 - sigmoid
// is.  sigmoid(l) / exp(high) = ex / (1 + exp(l)) loses none of a row's scores however small all of them are;
// where exp(high) is near fp32's end they are 1 / (1 + exp(-l)).  Quotients of 2 units of error, like their exponentials:
// full divisions, half a unit, take the forward 16.9 us for 15.1 and the gradient 10.8 for 9.9 (16384 tokens, 250 f32).
template <int V>
__device__ __forceinline__ void sigmoids(const float (&l)[V], const float (&ex)[V], float high, float (&score)[V],
                                         float (&off)[V]) {
  if (!(high > 60.f)) {
    const float scale = expf(high);
#pragma unroll
    for (int i = 0; i < V; ++i) off[i] = __fdividef(1.f, fmaf(ex[i], scale, 1.f)), score[i] = ex[i] * off[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float t = expf(-fabsf(l[i])), r = __fdividef(1.f, 1.f + t);
      score[i] = l[i] < 0.f ? t * r : r, off[i] = l[i] < 0.f ? r : t * r;
    }
  }
}

// Tokens whose rows a warp reads before it looks at any.
template <int V>
constexpr int kTokens = V <= 4 ? 4 : V <= 8 ? 2 : 1;

struct LossParams {
  const void* logits;
  int64_t ld, per_sequence;  // tokens of a sequence
  int32_t clusters, ctas;    // of a sequence; CTAs of a cluster
  int32_t run;               // tokens of a CTA
  int32_t experts, topk, slice;  // slice: experts that a CTA joins the sums of
  const int32_t* chosen;
  const uint8_t* mask;
  // of each cluster: sums of p [experts], counts [experts], {sum of lse^2, how many tokens count (an int)}
  float* sums;
  int32_t* run_counts;
  float2* rest;
  // where there is only one
  float* losses;
  int32_t* counts;
  int32_t* counted;
};

__device__ __forceinline__ void put_remote(const void* at, int rank, float v) {
  st_shared_cluster_u32(mapa_shared(smem_u32(at), uint32_t(rank)), __float_as_uint(v));
}
__device__ __forceinline__ void put_remote(const void* at, int rank, int v) {
  st_shared_cluster_u32(mapa_shared(smem_u32(at), uint32_t(rank)), uint32_t(v));
}

constexpr int kMaxCtas = 16;

// What the CTAs of a cluster hand to its first one.
struct Ends {
  float dot[kMaxCtas], z[kMaxCtas];
  int live[kMaxCtas], slots[kMaxCtas];
};

// Sums over the CTA's threads, in the same order each time; `part` is shared memory.  Thread 0 gets them.
__device__ __forceinline__ void block_sums(float& a, int& b, float2* part) {
  a = warp_sum(a), b = __reduce_add_sync(0xffffffffu, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __syncthreads();
  if (lane == 0) part[warp] = make_float2(a, __int_as_float(b));
  __syncthreads();
  if (threadIdx.x == 0) {
    a = 0.f, b = 0;
    for (int w = 0; w < warps; ++w) a += part[w].x, b += __float_as_int(part[w].y);
  }
}

template <int V, int UE, class T, bool kSigmoid>
__global__ void __launch_bounds__(32 * kWarps) balance_runs_kernel(LossParams p) {
  griddep_begin();
  p.logits = after_begin(p.logits), p.chosen = after_begin(p.chosen), p.mask = after_begin(p.mask);
  // [kWarps][experts] sums, [experts] counts; [ctas][slice] sums and counts for this CTA to join
  extern __shared__ float smem[];
  __shared__ float2 rest[kWarps];
  __shared__ Ends ends;
  int32_t* count = reinterpret_cast<int32_t*>(smem + kWarps * p.experts);
  float* join = reinterpret_cast<float*>(count + p.experts);
  int32_t* join_count = reinterpret_cast<int32_t*>(join + p.ctas * p.slice);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  const int64_t cluster = blockIdx.x / p.ctas;
  for (int e = threadIdx.x; e < p.experts; e += 32 * kWarps) count[e] = 0;
  __syncthreads();
  const int64_t sequence = cluster / p.clusters;
  const int64_t first = min((cluster - sequence * p.clusters) * p.ctas + rank, p.per_sequence) * p.run;
  const int n = int(max(int64_t(0), min(int64_t(p.run), p.per_sequence - first)));
  const int64_t t0 = sequence * p.per_sequence + first;
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  float z = 0.f;
  int live = 0;
  constexpr int U = kTokens<V>;
  for (int i0 = warp; i0 < n; i0 += U * kWarps) {  // U tokens side by side, for their latencies
    float l[U][V];
    int32_t chosen[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + i0 + u * kWarps;
      const bool on = i0 + u * kWarps < n && (p.mask == nullptr || p.mask[t] != 0);
      chosen[u] = -1;
      if (on) {
        load_row<V, UE, T>(static_cast<const T*>(p.logits) + t * p.ld, p.experts, l[u]);
        if (lane < p.topk) chosen[u] = __ldg(p.chosen + t * p.topk + lane);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[u][i] = -INFINITY;
      }
    }
    bool on[U];
    float high[U], total[U], score[kSigmoid ? U : 1][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      high[u] = row_max<V>(l[u]);
      on[u] = any_logit<V>(l[u], high[u]);
      if (on[u] && chosen[u] >= 0 && chosen[u] < p.experts) atomicAdd(count + chosen[u], 1);
      if constexpr (kSigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) score[u][i] = l[u][i];
      }
      total[u] = exponentials<V>(l[u], high[u]);  // of a token that does not count: NaN, and not used
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float lse = high[u] + logf(total[u]);
      z += on[u] ? lse * lse : 0.f, live += on[u] ? 1 : 0;
      float inv;
      if constexpr (kSigmoid) {
        float raw[V], off[V], all = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) raw[i] = score[u][i];
        sigmoids<V>(raw, l[u], high[u], score[u], off);
#pragma unroll
        for (int i = 0; i < V; ++i) all += score[u][i];
        inv = 1.f / warp_sum(all);
      } else {
        inv = 1.f / total[u];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += on[u] ? (kSigmoid ? score[kSigmoid ? u : 0][i] : l[u][i]) * inv : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (expert_of<UE>(i) < p.experts) smem[warp * p.experts + expert_of<UE>(i)] = sum[i];
  if (lane == 0) rest[warp] = make_float2(z, __int_as_float(live));
  __syncthreads();
  if (p.ctas > 1) cluster_sync();  // every CTA has started: its shared memory can be written
  for (int e = threadIdx.x; e < p.experts; e += 32 * kWarps) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += smem[w * p.experts + e];
    const int to = e / p.slice, at = rank * p.slice + e - to * p.slice;
    if (p.ctas > 1) {
      put_remote(join + at, to, s), put_remote(join_count + at, to, count[e]);
    } else {
      join[at] = s, join_count[at] = count[e];
    }
  }
  if (threadIdx.x == 0) {
    float zs = 0.f;
    int lives = 0;
    for (int w = 0; w < kWarps; ++w) zs += rest[w].x, lives += __float_as_int(rest[w].y);
    if (p.ctas > 1) {
      put_remote(ends.z + rank, 0, zs), put_remote(ends.live + rank, 0, lives);
    } else {
      ends.z[0] = zs, ends.live[0] = lives;
    }
  }
  __syncthreads();
  if (p.ctas > 1) cluster_sync();
  float dot = 0.f;
  int slots = 0;
  const int e0 = rank * p.slice;
  for (int i = threadIdx.x; i < min(p.slice, p.experts - e0); i += 32 * kWarps) {
    float s = 0.f;
    int c = 0;
    for (int r = 0; r < p.ctas; ++r) s += join[r * p.slice + i], c += join_count[r * p.slice + i];
    if (p.losses != nullptr) {
      p.counts[e0 + i] = c;
      dot += s * float(c), slots += c;
    } else {
      p.sums[cluster * p.experts + e0 + i] = s, p.run_counts[cluster * p.experts + e0 + i] = c;
    }
  }
  if (p.losses != nullptr) {
    block_sums(dot, slots, rest);
    if (p.ctas > 1) {
      if (threadIdx.x == 0) put_remote(ends.dot + rank, 0, dot), put_remote(ends.slots + rank, 0, slots);
      cluster_sync();
    } else if (threadIdx.x == 0) {
      ends.dot[0] = dot, ends.slots[0] = slots;
    }
  }
  if (rank == 0 && threadIdx.x == 0) {
    float zs = 0.f, dots = 0.f;
    int lives = 0, all = 0;
    for (int r = 0; r < p.ctas; ++r) {
      zs += ends.z[r], lives += ends.live[r];
      if (p.losses != nullptr) dots += ends.dot[r], all += ends.slots[r];
    }
    if (p.losses != nullptr) {
      const float tokens = float(max(lives, 1));
      p.losses[0] = all > 0 ? dots / float(all) * (float(p.experts) / tokens) : 0.f;
      p.losses[1] = zs / tokens;
      p.counted[0] = lives;
    } else {
      p.rest[cluster] = make_float2(zs, __int_as_float(lives));
    }
  }
}

struct JoinParams {
  const float* sums;
  const int32_t* run_counts;
  const float2* rest;
  int64_t sequences;
  int32_t clusters, experts, ctas;
  float* losses;
  int32_t* counts;
  int32_t* counted;
};

constexpr int kJoinWarps = 16, kJoinSequences = 64;

// Joins the clusters' sums: one cluster of its own.  CTAs take 64 sequences at a time, warps 32 experts of one.
__global__ void __launch_bounds__(32 * kJoinWarps) balance_join_kernel(JoinParams p) {
  griddep_begin();
  p.sums = after_begin(p.sums), p.run_counts = after_begin(p.run_counts), p.rest = after_begin(p.rest);
  __shared__ float2 part[kJoinWarps];
  __shared__ float dots[kJoinSequences][GMM_MAX_GROUPS / 32];
  __shared__ int slots[kJoinSequences][GMM_MAX_GROUPS / 32];
  __shared__ Ends ends;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.ctas > 1 ? int(cluster_ctarank()) : 0;
  float z = 0.f;
  int live = 0;
  for (int64_t c = int64_t(rank) * 32 * kJoinWarps + threadIdx.x; c < p.sequences * p.clusters;
       c += int64_t(p.ctas) * 32 * kJoinWarps) {
    const float2 r = __ldg(p.rest + c);
    z += r.x, live += __float_as_int(r.y);
  }
  const int segments = (p.experts + 31) / 32;
  const int64_t each = (p.sequences + p.ctas - 1) / p.ctas;  // sequences of a CTA
  const int64_t s0 = min(each * rank, p.sequences), s1 = min(s0 + each, p.sequences);
  float balance = 0.f;
  for (int64_t first = s0; first < s1; first += kJoinSequences) {
    const int n = int(min(s1 - first, int64_t(kJoinSequences)));
    for (int i = warp; i < n * segments; i += kJoinWarps) {
      const int s = i / segments, e = (i - s * segments) * 32 + lane;
      float sum = 0.f;
      int count = 0;
      if (e < p.experts) {
        const int64_t at = (first + s) * p.clusters * p.experts + e;
#pragma unroll 8
        for (int c = 0; c < p.clusters; ++c) {
          sum += __ldg(p.sums + at + int64_t(c) * p.experts), count += __ldg(p.run_counts + at + int64_t(c) * p.experts);
        }
        p.counts[(first + s) * p.experts + e] = count;
      }
      sum = warp_sum(sum * float(count)), count = __reduce_add_sync(0xffffffffu, count);
      if (lane == 0) dots[s][i - s * segments] = sum, slots[s][i - s * segments] = count;
    }
    __syncthreads();
    if (threadIdx.x < n) {
      float dot = 0.f;
      int all = 0;
      for (int g = 0; g < segments; ++g) dot += dots[threadIdx.x][g], all += slots[threadIdx.x][g];
      if (all > 0) balance += dot / float(all);
    }
    __syncthreads();
  }
  int none = 0;
  block_sums(balance, none, part);
  block_sums(z, live, part);
  if (p.ctas > 1) cluster_sync();
  if (threadIdx.x == 0) {
    if (p.ctas > 1) {
      put_remote(ends.dot + rank, 0, balance), put_remote(ends.z + rank, 0, z), put_remote(ends.slots + rank, 0, live);
    } else {
      ends.dot[0] = balance, ends.z[0] = z, ends.slots[0] = live;
    }
  }
  if (p.ctas > 1) cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    balance = 0.f, z = 0.f, live = 0;
    for (int r = 0; r < p.ctas; ++r) balance += ends.dot[r], z += ends.z[r], live += ends.slots[r];
    const float n = float(max(live, 1));
    p.losses[0] = balance * (float(p.experts) / n);
    p.losses[1] = z / n;
    p.counted[0] = live;
  }
}

struct BackParams {
  const float* dlosses;
  const int32_t* counts;
  const int32_t* counted;
  const void* logits;
  int64_t tokens, ld, per_sequence;
  int32_t experts, run;  // tokens of a warp, consecutive ones
  const uint8_t* mask;
  void* dlogits;
};

// A warp a token, some tokens one after another.
template <int V, int UE, class T, bool kSigmoid>
__global__ void __launch_bounds__(32 * kBackWarps) balance_backward_kernel(BackParams p) {
  griddep_begin();
  p.dlosses = after_begin(p.dlosses), p.counts = after_begin(p.counts), p.counted = after_begin(p.counted);
  p.logits = after_begin(p.logits), p.mask = after_begin(p.mask);
  const int64_t t0 = (int64_t(blockIdx.x) * kBackWarps + (threadIdx.x >> 5)) * p.run;
  const int n = int(min(int64_t(p.run), p.tokens - t0));
  const float tokens = float(max(p.counted[0], 1));
  const float per_token = p.dlosses[0] * (float(p.experts) / tokens), d1 = 2.f * p.dlosses[1] / tokens;
  float share[V], d0 = 0.f;  // of the sequence: counts, and what takes them to shares
  int64_t left = 0, sequence = -1;  // tokens of the sequence still to come
  constexpr int U = V <= 4 ? 2 : 1;
  for (int i0 = 0; i0 < n; i0 += U) {
    float l[U][V];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + i0 + u;
      on[u] = i0 + u < n && (p.mask == nullptr || p.mask[t] != 0);
      if (on[u]) load_row<V, UE, T>(static_cast<const T*>(p.logits) + t * p.ld, p.experts, l[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + i0 + u;
      if (i0 + u >= n) break;
      if (left == 0) {
        sequence = sequence < 0 ? t / p.per_sequence : sequence + 1;
        left = (sequence + 1) * p.per_sequence - t;
        int slots = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = expert_of<UE>(i) < p.experts ? __ldg(p.counts + sequence * p.experts + expert_of<UE>(i)) : 0;
          slots += c, share[i] = float(c);
        }
        d0 = per_token / float(max(__reduce_add_sync(0xffffffffu, slots), 1));
      }
      --left;
      float d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.f;
      const float high = on[u] ? row_max<V>(l[u]) : 0.f;
      if (on[u] && any_logit<V>(l[u], high)) {
        float score[V], off[V];
        if constexpr (kSigmoid) {
#pragma unroll
          for (int i = 0; i < V; ++i) score[i] = l[u][i];
        }
        float total = exponentials<V>(l[u], high);
        const float zf = d1 * (high + logf(total)) / total;
        if constexpr (kSigmoid) {
          float raw[V];
#pragma unroll
          for (int i = 0; i < V; ++i) raw[i] = score[i];
          sigmoids<V>(raw, l[u], high, score, off);
          total = 0.f;
#pragma unroll
          for (int i = 0; i < V; ++i) total += score[i];
          total = warp_sum(total);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) score[i] = l[u][i];
        }
        const float inv = 1.f / total;
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) mean += share[i] * (score[i] * inv);
        mean = warp_sum(mean);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float q = d0 * (score[i] * inv) * (share[i] - mean);
          d[i] = (kSigmoid ? q * off[i] : q) + zf * l[u][i];
        }
      }
      T* out = static_cast<T*>(p.dlogits) + t * p.experts;
#pragma unroll
      for (int i = 0; i < V; i += UE) {
        const int e = expert_of<UE>(i);
        if (e >= p.experts) continue;
        using Bits = std::conditional_t<sizeof(T) * UE == 16, uint4, std::conditional_t<sizeof(T) * UE == 8, uint2,
                     std::conditional_t<sizeof(T) * UE == 4, uint32_t, uint16_t>>>;
        Bits bits;
#pragma unroll
        for (int j = 0; j < UE; ++j) put(reinterpret_cast<T*>(&bits) + j, d[i + j]);
        *reinterpret_cast<Bits*>(out + e) = bits;
      }
    }
  }
}

int lane_experts(int experts) {
  int v = 1;
  while (v * 32 < experts) v *= 2;
  return v;
}

template <class F>
cudaError_t by_width(int v, F&& go) {
  switch (v) {
    case 1: return go(std::integral_constant<int, 1>{});
    case 2: return go(std::integral_constant<int, 2>{});
    case 4: return go(std::integral_constant<int, 4>{});
    case 8: return go(std::integral_constant<int, 8>{});
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
  }
  return cudaErrorInvalidValue;
}

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// How the tokens are cut up: CTAs of a cluster, clusters of a sequence, tokens of a CTA.
struct Cut {
  int ctas;
  int64_t clusters, run;
};
// A CTA has two tokens for each of its warps; all of them are about kCtas, or one cluster where its
// warps have at most eight (512 tokens 5.3 us, in two kernels 6.9; 1024: 5.8 and 8.0; 2048: 8.0 and 8.6; 4096:
// 12.0 and 9.8).
Cut cut_of(int64_t tokens, int64_t sequences) {
  const int64_t per = tokens / sequences;
  Cut c{1, 1, per > 0 ? per : 1};
  if (per == 0) return c;
  const int64_t wanted = (per + 2 * kWarps - 1) / (2 * kWarps);  // CTAs of a sequence, were there no others
  const int64_t share = sequences < kCtas ? kCtas / sequences : 1;
  int64_t ctas = wanted < share ? wanted : share;
  if (sequences == 1 && tokens <= 8 * kWarps * kMaxCtas && ctas > kMaxCtas) ctas = kMaxCtas;
  c.ctas = sequences == 1 && ctas == kMaxCtas ? kMaxCtas : ctas >= 8 ? 8 : ctas >= 4 ? 4 : ctas >= 2 ? 2 : 1;
  c.clusters = ctas / c.ctas;
  const int64_t all = c.clusters * c.ctas;
  c.run = (per + all - 1) / all;
  return c;
}

bool sizes_ok(int64_t tokens, int32_t experts, int64_t sequences) {
  return tokens >= 0 && experts >= 1 && experts <= GMM_MAX_GROUPS && sequences >= 1 && tokens <= kMaxSize &&
         sequences <= kMaxSize && tokens % sequences == 0;
}

int check(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld, int score, int64_t sequences) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (!sizes_ok(tokens, experts, sequences) || ld < experts) return GMM_ERR_SHAPE;
  if (score != GMM_SCORE_SOFTMAX && score != GMM_SCORE_SIGMOID) return GMM_ERR_SHAPE;
  if (misaligned(logits, dtype == GMM_DTYPE_F32 ? 4 : 2)) return GMM_ERR_ALIGN;
  return GMM_OK;
}

template <class K>
cudaError_t allow_16(K kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

template <class T>
cudaError_t balance_runs(const LossParams& p, bool sigmoid, int64_t ctas, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value, W = kUnit<V, T>;
    const bool wide = p.experts % W == 0 && p.ld % W == 0 && !misaligned(p.logits, W * sizeof(T));
    auto kern = wide ? (sigmoid ? balance_runs_kernel<V, W, T, true> : balance_runs_kernel<V, W, T, false>)
                     : (sigmoid ? balance_runs_kernel<V, 1, T, true> : balance_runs_kernel<V, 1, T, false>);
    if (p.ctas > 8)
      if (cudaError_t e = allow_16(kern)) return e;
    const size_t smem = (size_t(kWarps + 1) * p.experts + 2 * size_t(p.ctas) * p.slice) * 4;
    // past 40 KB the kernel's limit is raised, to one size for all calls: that of the most experts
    constexpr size_t kMost = (size_t(kWarps + 1) * GMM_MAX_GROUPS + 2 * (GMM_MAX_GROUPS + kMaxCtas)) * 4;
    if (smem > 40 * 1024)
      if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost))) return e;
    return launch_dependent(kern, unsigned(ctas), 32 * kWarps, smem, stream, p.ctas, p);
  });
}

template <class T>
cudaError_t balance_backward(const BackParams& p, bool sigmoid, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value, W = kUnit<V, T>;
    const bool wide = p.experts % W == 0 && p.ld % W == 0 && !misaligned(p.logits, W * sizeof(T)) &&
                      !misaligned(p.dlogits, W * sizeof(T));
    auto kern = wide ? (sigmoid ? balance_backward_kernel<V, W, T, true> : balance_backward_kernel<V, W, T, false>)
                     : (sigmoid ? balance_backward_kernel<V, 1, T, true> : balance_backward_kernel<V, 1, T, false>);
    const int64_t per_cta = int64_t(p.run) * kBackWarps;
    return launch_dependent(kern, unsigned((p.tokens + per_cta - 1) / per_cta), 32 * kBackWarps, 0, stream, 1, p);
  });
}

}  // namespace
}  // namespace gmmk

extern "C" size_t gmm_balance_scratch_bytes(int64_t tokens, int32_t num_experts, int64_t sequences) {
  using namespace gmmk;
  if (!sizes_ok(tokens, num_experts, sequences)) return 0;
  const int64_t clusters = sequences * cut_of(tokens, sequences).clusters;
  if (clusters == 1) return 0;
  return size_t(clusters) * (size_t(num_experts) * 8 + 8) + 16;
}

extern "C" int gmm_balance_loss(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts,
                                int64_t logits_ld, const int32_t* experts, int32_t topk, int score,
                                const uint8_t* token_mask, int64_t sequences, float* losses, int32_t* counts,
                                int32_t* counted, void* scratch, size_t scratch_bytes, void* stream) {
  using namespace gmmk;
  if (int st = check(logits, logits_dtype, tokens, num_experts, logits_ld, score, sequences)) return st;
  if (topk < 1 || topk > GMM_MAX_TOPK || tokens * topk > kMaxSize) return GMM_ERR_SHAPE;
  if ((tokens > 0 && (logits == nullptr || experts == nullptr)) || losses == nullptr || counts == nullptr ||
      counted == nullptr)
    return GMM_ERR_NULL;
  if (misaligned(experts, 4) || misaligned(losses, 4) || misaligned(counts, 4) || misaligned(counted, 4) ||
      misaligned(scratch, 16))
    return GMM_ERR_ALIGN;
  const size_t needed = gmm_balance_scratch_bytes(tokens, num_experts, sequences);
  if (scratch_bytes < needed || (needed > 0 && scratch == nullptr)) return GMM_ERR_WORKSPACE;
  if (int st = require_device(nullptr)) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Cut cut = cut_of(tokens, sequences);
  const int64_t clusters = sequences * cut.clusters;
  float2* rest = static_cast<float2*>(scratch);
  float* sums = reinterpret_cast<float*>(rest + clusters);
  int32_t* run_counts = reinterpret_cast<int32_t*>(sums + clusters * num_experts);
  LossParams p{logits, logits_ld, tokens / sequences, int32_t(cut.clusters), cut.ctas, int32_t(cut.run), num_experts, topk,
               (num_experts + cut.ctas - 1) / cut.ctas, experts, token_mask, sums, run_counts, rest, nullptr, nullptr,
               nullptr};
  if (clusters == 1) p.losses = losses, p.counts = counts, p.counted = counted;
  const bool sig = score == GMM_SCORE_SIGMOID;
  cudaError_t e = logits_dtype == GMM_DTYPE_F32 ? balance_runs<float>(p, sig, clusters * cut.ctas, s)
                                                : balance_runs<__nv_bfloat16>(p, sig, clusters * cut.ctas, s);
  if (e == cudaSuccess && clusters > 1) {
    // two turns of a CTA's warps, on up to 16 CTAs
    const int64_t turns = sequences * ((num_experts + 31) / 32);
    int ctas = 1;
    while (ctas < kMaxCtas && ctas * 2 <= sequences && ctas * 2 * kJoinWarps < turns) ctas *= 2;
    const JoinParams j{sums, run_counts, rest, sequences, int32_t(cut.clusters), num_experts, ctas, losses, counts,
                       counted};
    if (ctas > 8) e = allow_16(balance_join_kernel);
    if (e == cudaSuccess) e = launch_dependent(balance_join_kernel, unsigned(ctas), 32 * kJoinWarps, 0, s, ctas, j);
  }
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}

extern "C" int gmm_balance_loss_backward(const float* dlosses, const int32_t* counts, const int32_t* counted,
                                         const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts,
                                         int64_t logits_ld, int score, const uint8_t* token_mask, int64_t sequences,
                                         void* dlogits, void* stream) {
  using namespace gmmk;
  if (int st = check(logits, logits_dtype, tokens, num_experts, logits_ld, score, sequences)) return st;
  if (tokens > 0 && (dlosses == nullptr || counts == nullptr || counted == nullptr || logits == nullptr ||
                     dlogits == nullptr))
    return GMM_ERR_NULL;
  if (misaligned(dlosses, 4) || misaligned(counts, 4) || misaligned(counted, 4) ||
      misaligned(dlogits, logits_dtype == GMM_DTYPE_F32 ? 4 : 2))
    return GMM_ERR_ALIGN;
  int sms = 0;
  if (int st = require_device(&sms)) return st;
  if (tokens == 0) return GMM_OK;
  // tokens of a warp: one while all warps fit the GPU at once
  int64_t run = tokens / (int64_t(sms) * 6 * kBackWarps);
  run = run < 1 ? 1 : run > 8 ? 8 : run;
  const BackParams p{dlosses, counts, counted, logits, tokens, logits_ld, tokens / sequences, num_experts, int32_t(run),
                     token_mask, dlogits};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sig = score == GMM_SCORE_SIGMOID;
  const cudaError_t e =
      logits_dtype == GMM_DTYPE_F32 ? balance_backward<float>(p, sig, s) : balance_backward<__nv_bfloat16>(p, sig, s);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
