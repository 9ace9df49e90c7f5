// The losses that keep a router's experts evenly loaded, with the experts' loads,
// and the gradient of the losses with respect to the logits.
//
//   p[t]   softmax of token t's logits, or their sigmoids over the sum of these
//   f[s]   shares of sequence s's slots that each expert got (no gradient)
//   balance = E/N sum_t <f[s(t)], p[t]>        z = 1/N sum_t lse(l[t])^2
//   dl = d0 E/N p (f - <f, p>) + d1 2/N lse softmax(l)
// and with sigmoid scores the first term times 1 - sigmoid(l).  Normalised
// sigmoids are a softmax of log sigmoid(l), which neither overflows nor loses
// tiny scores.  f is known only when all tokens have been counted, but
// sum_t <f, p[t]> = <f, sum_t p[t]>: one pass over the logits sums p by expert.
//
// Forward: CTAs sum p, lse^2 and the counts of a run of tokens of one sequence (a
// warp a token, a lane V consecutive experts, sums in registers), and a second
// kernel, one cluster, joins the runs in their order.
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// V consecutive logits of this lane (past the last expert: -inf), in whole 16-byte
// loads where the rows allow them.
template <int V, class T>
__device__ __forceinline__ void load_row(const T* row, int e0, int experts, bool wide, float (&l)[V]) {
  constexpr int kBytes = V * int(sizeof(T));
  if constexpr (kBytes % 16 == 0) {
    if (wide) {  // experts % V == 0: the lane's V are all there or none is
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = -INFINITY;
      if (e0 < experts) {
        uint4 raw[kBytes / 16];
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
        const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = as_float(t[i]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? as_float(row[e0 + i]) : -INFINITY;
}

// l becomes exp(l - max), unnormalised; returns its sum over the warp's row, with the maximum.
template <int V>
__device__ __forceinline__ float exponentials(float (&l)[V], float& high) {
  high = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) high = fmaxf(high, l[i]);
  high = warp_max(high);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += l[i] = expf(l[i] - high);
  return warp_sum(sum);
}

// Whether a row has anything but -inf (NaN counts as something).
template <int V>
__device__ __forceinline__ bool any_logit(const float (&l)[V]) {
  bool some = false;
#pragma unroll
  for (int i = 0; i < V; ++i) some |= l[i] != -INFINITY;
  return __any_sync(0xffffffffu, some);
}

struct LossParams {
  const void* logits;
  int64_t ld, per_sequence, runs_per_sequence, run;  // tokens of a sequence, its runs, tokens of a run
  int32_t experts, topk, wide;
  const int32_t* chosen;
  const uint8_t* mask;
  // of each run: sums of p [experts], counts [experts], {sum of lse^2, tokens that count}
  float* sums;
  int32_t* counts;
  float2* rest;
};

// One CTA a run.
template <int V, class T, bool kSigmoid>
__global__ void __launch_bounds__(32 * kWarps) balance_runs_kernel(LossParams p) {
  griddep_begin();
  p.logits = after_begin(p.logits), p.chosen = after_begin(p.chosen), p.mask = after_begin(p.mask);
  extern __shared__ float smem[];  // [kWarps][experts] sums, then [experts] counts
  __shared__ float2 rest[kWarps];
  int32_t* count = reinterpret_cast<int32_t*>(smem + kWarps * p.experts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e0 = lane * V;
  for (int e = threadIdx.x; e < p.experts; e += 32 * kWarps) count[e] = 0;
  __syncthreads();
  const int64_t sequence = blockIdx.x / p.runs_per_sequence, run = blockIdx.x % p.runs_per_sequence;
  const int64_t first = run * p.run, n = min(p.run, p.per_sequence - first);
  const int64_t t0 = sequence * p.per_sequence + first;
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  float z = 0.f, live = 0.f;
  for (int64_t i = warp; i < n; i += kWarps) {
    const int64_t t = t0 + i;
    if (p.mask != nullptr && p.mask[t] == 0) continue;
    float l[V];
    load_row<V, T>(static_cast<const T*>(p.logits) + t * p.ld, e0, p.experts, p.wide != 0, l);
    const int32_t e = lane < p.topk ? p.chosen[t * p.topk + lane] : -1;
    if (!any_logit<V>(l)) continue;
    if (e >= 0 && e < p.experts) atomicAdd(count + e, 1);
    float v[V], high;
    if constexpr (kSigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = log_sigmoid(l[i]);
    }
    float total = exponentials<V>(l, high);
    const float lse = high + logf(total);
    z += lse * lse;
    live += 1.f;
    if constexpr (kSigmoid) total = exponentials<V>(v, high);
    const float inv = 1.f / total;
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += (kSigmoid ? v[i] : l[i]) * inv;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < p.experts) smem[warp * p.experts + e0 + i] = sum[i];
  if (lane == 0) rest[warp] = make_float2(z, live);
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += 32 * kWarps) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += smem[w * p.experts + e];
    p.sums[int64_t(blockIdx.x) * p.experts + e] = s;
    p.counts[int64_t(blockIdx.x) * p.experts + e] = count[e];
  }
  if (threadIdx.x == 0) {
    float2 r = rest[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) r.x += rest[w].x, r.y += rest[w].y;
    p.rest[blockIdx.x] = r;
  }
}

struct JoinParams {
  const float* sums;
  const int32_t* run_counts;
  const float2* rest;
  int64_t sequences, runs_per_sequence;
  int32_t experts;
  float* losses;
  int32_t* counts;
  int32_t* counted;
};

constexpr int kJoinThreads = 512;

// Joins the runs: one CTA.
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(JoinParams p) {
  griddep_begin();
  p.sums = after_begin(p.sums), p.run_counts = after_begin(p.run_counts), p.rest = after_begin(p.rest);
  __shared__ float part[3][kJoinThreads / 32];
  __shared__ int part_n[kJoinThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarpsHere = kJoinThreads / 32;
  float balance = 0.f;
  for (int64_t s = 0; s < p.sequences; ++s) {
    const int64_t r0 = s * p.runs_per_sequence;
    float dot = 0.f;
    int slots = 0;
    for (int e = threadIdx.x; e < p.experts; e += kJoinThreads) {
      float sum = 0.f;
      int n = 0;
      for (int64_t r = r0; r < r0 + p.runs_per_sequence; ++r)
        sum += p.sums[r * p.experts + e], n += p.run_counts[r * p.experts + e];
      p.counts[s * p.experts + e] = n;
      dot += sum * float(n), slots += n;
    }
    dot = warp_sum(dot), slots = __reduce_add_sync(0xffffffffu, slots);
    __syncthreads();
    if (lane == 0) part[0][warp] = dot, part_n[warp] = slots;
    __syncthreads();
    if (threadIdx.x == 0) {
      float d = 0.f;
      int n = 0;
      for (int w = 0; w < kWarpsHere; ++w) d += part[0][w], n += part_n[w];
      if (n > 0) balance += d / float(n);
    }
  }
  float z = 0.f;
  int live = 0;
  for (int64_t r = threadIdx.x; r < p.sequences * p.runs_per_sequence; r += kJoinThreads)
    z += p.rest[r].x, live += int(p.rest[r].y);
  z = warp_sum(z), live = __reduce_add_sync(0xffffffffu, live);
  __syncthreads();
  if (lane == 0) part[1][warp] = z, part_n[warp] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    z = 0.f, live = 0;
    for (int w = 0; w < kWarpsHere; ++w) z += part[1][w], live += part_n[w];
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
  int32_t experts, wide;
  const uint8_t* mask;
  void* dlogits;
};

// A warp a token.
template <int V, class T, bool kSigmoid>
__global__ void __launch_bounds__(32 * kWarps) balance_backward_kernel(BackParams p) {
  griddep_begin();
  p.dlosses = after_begin(p.dlosses), p.counts = after_begin(p.counts), p.counted = after_begin(p.counted);
  p.logits = after_begin(p.logits), p.mask = after_begin(p.mask);
  const int lane = threadIdx.x & 31, e0 = lane * V;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = 0.f;
  if (p.mask == nullptr || p.mask[t] != 0) {
    float l[V];
    load_row<V, T>(static_cast<const T*>(p.logits) + t * p.ld, e0, p.experts, p.wide != 0, l);
    if (any_logit<V>(l)) {
      const int32_t* counts = p.counts + (t / p.per_sequence) * p.experts;
      float share[V];
      int slots = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int n = e0 + i < p.experts ? counts[e0 + i] : 0;
        slots += n, share[i] = float(n);
      }
      slots = __reduce_add_sync(0xffffffffu, slots);
      const float n = float(max(p.counted[0], 1));
      const float d0 = p.dlosses[0] * (float(p.experts) / n) / float(max(slots, 1)), d1 = 2.f * p.dlosses[1] / n;
      float v[V], off[V], high;
      if constexpr (kSigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = log_sigmoid(l[i]), off[i] = 1.f / (1.f + expf(l[i]));
      }
      float total = exponentials<V>(l, high);
      const float zf = d1 * (high + logf(total)) / total;
      if constexpr (kSigmoid) total = exponentials<V>(v, high);
      const float inv = 1.f / total;
      float mean = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) mean += share[i] * ((kSigmoid ? v[i] : l[i]) * inv);
      mean = warp_sum(mean);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float q = d0 * ((kSigmoid ? v[i] : l[i]) * inv) * (share[i] - mean);
        d[i] = (kSigmoid ? q * off[i] : q) + zf * l[i];
      }
    }
  }
  T* out = static_cast<T*>(p.dlogits) + t * p.experts;
  constexpr int kBytes = V * int(sizeof(T));
  if constexpr (kBytes % 16 == 0) {
    if (p.wide) {
      if (e0 < p.experts) {
        uint4 raw[kBytes / 16];
        T* o = reinterpret_cast<T*>(raw);
#pragma unroll
        for (int i = 0; i < V; ++i) put(o + i, d[i]);
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(out + e0)[i] = raw[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < p.experts) put(out + e0 + i, d[i]);
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

// Tokens of a run: some 300 runs in all, of whole warps' turns.
int64_t run_of(int64_t tokens, int64_t per_sequence) {
  int64_t run = (tokens / 304 + kWarps - 1) / kWarps * kWarps;
  if (run < 4 * kWarps) run = 4 * kWarps;
  return run < per_sequence ? run : (per_sequence > 0 ? per_sequence : 1);
}
int64_t runs_of(int64_t per_sequence, int64_t run) { return (per_sequence + run - 1) / run; }

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

template <class T>
cudaError_t balance_runs(LossParams p, bool sigmoid, int64_t runs, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value;
    p.wide = p.experts % V == 0 && p.ld * sizeof(T) % 16 == 0 && !misaligned(p.logits, 16);
    auto kern = sigmoid ? balance_runs_kernel<V, T, true> : balance_runs_kernel<V, T, false>;
    return launch_dependent(kern, unsigned(runs), 32 * kWarps, size_t(kWarps + 1) * p.experts * 4, stream, 1, p);
  });
}

template <class T>
cudaError_t balance_backward(BackParams p, bool sigmoid, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value;
    p.wide = p.experts % V == 0 && p.ld * sizeof(T) % 16 == 0 && !misaligned(p.logits, 16) &&
             p.experts * sizeof(T) % 16 == 0 && !misaligned(p.dlogits, 16);
    auto kern = sigmoid ? balance_backward_kernel<V, T, true> : balance_backward_kernel<V, T, false>;
    return launch_dependent(kern, unsigned((p.tokens + kWarps - 1) / kWarps), 32 * kWarps, 0, stream, 1, p);
  });
}

}  // namespace
}  // namespace gmmk

extern "C" size_t gmm_balance_scratch_bytes(int64_t tokens, int32_t num_experts, int64_t sequences) {
  using namespace gmmk;
  if (!sizes_ok(tokens, num_experts, sequences)) return 0;
  const int64_t runs = sequences * runs_of(tokens / sequences, run_of(tokens, tokens / sequences));
  return size_t(runs) * (size_t(num_experts) * 8 + 8) + 16;
}

extern "C" int gmm_balance_loss(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts,
                                int64_t logits_ld, const int32_t* experts, int32_t topk, int score,
                                const uint8_t* token_mask, int64_t sequences, float* losses, int32_t* counts,
                                int32_t* counted, void* scratch, size_t scratch_bytes, void* stream) {
  using namespace gmmk;
  if (int st = check(logits, logits_dtype, tokens, num_experts, logits_ld, score, sequences)) return st;
  if (topk < 1 || topk > GMM_MAX_TOPK || tokens * topk > kMaxSize) return GMM_ERR_SHAPE;
  if ((tokens > 0 && (logits == nullptr || experts == nullptr)) || losses == nullptr || counts == nullptr ||
      counted == nullptr || scratch == nullptr)
    return GMM_ERR_NULL;
  if (misaligned(experts, 4) || misaligned(losses, 4) || misaligned(counts, 4) || misaligned(counted, 4) ||
      misaligned(scratch, 16))
    return GMM_ERR_ALIGN;
  if (scratch_bytes < gmm_balance_scratch_bytes(tokens, num_experts, sequences)) return GMM_ERR_WORKSPACE;
  if (int st = require_device(nullptr)) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t per = tokens / sequences, run = run_of(tokens, per), each = runs_of(per, run), runs = sequences * each;
  float2* rest = static_cast<float2*>(scratch);
  float* sums = reinterpret_cast<float*>(rest + runs);
  int32_t* run_counts = reinterpret_cast<int32_t*>(sums + runs * num_experts);
  cudaError_t e = cudaSuccess;
  if (tokens > 0) {
    const LossParams p{logits, logits_ld, per, each, run, num_experts, topk, 0, experts, token_mask, sums, run_counts,
                       rest};
    const bool sig = score == GMM_SCORE_SIGMOID;
    e = logits_dtype == GMM_DTYPE_F32 ? balance_runs<float>(p, sig, runs, s) : balance_runs<__nv_bfloat16>(p, sig, runs, s);
  }
  if (e == cudaSuccess) {
    const JoinParams p{sums, run_counts, rest, sequences, each, num_experts, losses, counts, counted};
    e = launch_dependent(balance_join_kernel, 1, kJoinThreads, 0, s, 1, p);
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
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const BackParams p{dlosses, counts, counted, logits, tokens, logits_ld, tokens / sequences, num_experts, 0,
                     token_mask, dlogits};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sig = score == GMM_SCORE_SIGMOID;
  const cudaError_t e =
      logits_dtype == GMM_DTYPE_F32 ? balance_backward<float>(p, sig, s) : balance_backward<__nv_bfloat16>(p, sig, s);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
