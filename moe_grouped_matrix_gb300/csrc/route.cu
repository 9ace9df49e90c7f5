// The router of a mixture-of-experts layer: the top-k choice of experts with
// its weights, and the gradient of the weights with respect to the logits.
//
//   key[e] = l[e] + bias[e], or s(l)[e] + bias[e];  chosen: the topk largest keys, ties by index
//   w_j = scale * s(l)[e_j], or scale * s(l)[e_j] / sum_i s(l)[e_i]
// with s the softmax over all experts or the sigmoid.  Renormalised weights of
// either score are a softmax over the chosen experts' values v, v = l for the
// softmax (the sum over all experts cancels) and v = log sigmoid(l) for the
// sigmoid, which neither overflows nor loses tiny scores.
//
// One warp per token; lane i holds the V consecutive experts from i * V, so
// that equal keys are ordered by lane first.  A key is mapped to an unsigned
// integer with the same order (0: cannot be chosen) and each of the topk rounds
// is one warp-wide integer maximum, a ballot for the lowest lane that holds it
// and a rescan of that lane's V keys.  Bound by the rounds' latency: 64 tokens, 4
// of 64 experts, 1.7 us in a graph; 4096 tokens, 8 of 128 experts, 5.4 us for 1 or
// 2 MB of logits, 5.6 with a bias on the logits and 6.5 with one on the scores, whose
// exponentials come before the choice (a kernel of its own: as a branch in one
// kernel it took the other forms 6.0 us).
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// An unsigned integer ordered as the key; 0 for a key that cannot be chosen.
__device__ __forceinline__ uint32_t ordered(float key) {
  const uint32_t b = __float_as_uint(key + 0.f);  // -0 counts as 0
  if (!(key > -INFINITY)) return 0u;              // -inf or NaN
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

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

__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l));  // neither side overflows
  return (l < 0.f ? e : 1.f) / (1.f + e);
}
__device__ __forceinline__ float log_sigmoid(float l) { return fminf(l, 0.f) - log1pf(expf(-fabsf(l))); }

// V consecutive logits of this lane (past the last expert: -inf).  Whole 16-byte
// loads where the rows allow them.
template <int V, class T>
__device__ __forceinline__ void load_row(const T* row, int e0, int experts, bool wide, float (&l)[V]) {
  constexpr int kBytes = V * int(sizeof(T));
  if (kBytes % 16 == 0 && wide) {
    if constexpr (kBytes % 16 == 0) {
      if (e0 < experts) {  // wide: experts % V == 0, so the lane's V are all there or none is
        uint4 raw[kBytes / 16];
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row + e0) + i);
        const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = float(t[i]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) l[i] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? load_logit(row + e0 + i) : -INFINITY;
  }
}

struct RouteParams {
  const void* logits;
  int64_t tokens, ld;
  int32_t experts, topk;
  int32_t sigmoid, renormalize, wide;
  float scale;
  const float* bias;
  const uint8_t* mask;
  float* weights;
  int32_t* chosen;
};

// kScored: the bias is the score's.
template <int V, class T, bool kScored>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteParams p) {
  griddep_begin();
  p.logits = after_begin(p.logits), p.bias = after_begin(p.bias), p.mask = after_begin(p.mask);
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const bool live = p.mask == nullptr || p.mask[t] != 0;
  const int e0 = lane * V;
  float l[V];
  uint32_t key[V];
  if (live) {
    load_row<V, T>(static_cast<const T*>(p.logits) + t * p.ld, e0, p.experts, p.wide != 0, l);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = -INFINITY;
  }
  // The softmax over all experts is exp(l - high) / total.
  auto over_all = [&](float& high, float& total) {
    high = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) high = fmaxf(high, l[i]);
    high = warp_max(high);
#pragma unroll
    for (int i = 0; i < V; ++i) total += expf(l[i] - high);
    total = warp_sum(total);
  };
  float high = 0.f, total = 1.f;
  if (kScored && !p.sigmoid) over_all(high, total);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float b = p.bias != nullptr && e0 + i < p.experts ? __ldg(p.bias + e0 + i) : 0.f;
    float to = l[i];
    if constexpr (kScored) {
      if (to > -INFINITY) to = p.sigmoid ? sigmoid(to) : expf(to - high) / total;
    }
    key[i] = ordered(to + b);
  }
  uint32_t best = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (key[i] > best) best = key[i], at = i;

  int32_t mine = -1;        // the expert of slot `lane`
  float mine_l = -INFINITY; // and its logit
  for (int j = 0; j < p.topk; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0) break;
    const int w = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    float lw = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i == at) lw = l[i];
    const int ew = __shfl_sync(0xffffffffu, e0 + at, w);
    lw = __shfl_sync(0xffffffffu, lw, w);
    if (lane == j) mine = ew, mine_l = lw;
    if (lane == w) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = 0;
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] > best) best = key[i], at = i;
    }
  }
  const bool took = mine >= 0;
  const float v = p.sigmoid ? log_sigmoid(mine_l) : mine_l;
  float w = 0.f;
  if (p.renormalize) {
    const float top = warp_max(took ? v : -INFINITY);
    const float e = took ? expf(v - top) : 0.f;
    const float sum = warp_sum(e);
    w = took ? p.scale * (e / sum) : 0.f;
  } else if (p.sigmoid) {
    w = took ? p.scale * expf(v) : 0.f;
  } else if (live) {
    if (!kScored) over_all(high, total);
    w = took ? p.scale * (expf(mine_l - high) / total) : 0.f;
  }
  if (lane < p.topk) {
    p.weights[t * p.topk + lane] = w;
    p.chosen[t * p.topk + lane] = mine;
  }
}

struct RouteBackParams {
  const float* dweights;
  const int32_t* chosen;
  const void* logits;
  int64_t tokens, ld;
  int32_t experts, topk;
  int32_t sigmoid, renormalize, wide;
  float scale;
  void* dlogits;
};

// dl from g_j = scale * dw_j, with w'_j the weights without scale:
//   renormalised   dv_j = w'_j (g_j - sum_i g_i w'_i)
//   softmax        dl_e = p_e (g_e - sum_i g_i p_{e_i}),  g_e = 0 where not chosen
//   sigmoid        dl_j = w'_j (1 - sigmoid(l_j)) g_j
// and dl_j = dv_j (1 - sigmoid(l_j)) for the renormalised sigmoid.
template <int V, class T>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(RouteBackParams p) {
  griddep_begin();
  p.dweights = after_begin(p.dweights), p.chosen = after_begin(p.chosen), p.logits = after_begin(p.logits);
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  const int e0 = lane * V;
  const bool slot = lane < p.topk;
  const int32_t e = slot ? p.chosen[t * p.topk + lane] : -1;
  const bool took = e >= 0 && e < p.experts;
  const float g = took ? p.scale * p.dweights[t * p.topk + lane] : 0.f;
  const float le = took ? load_logit(row + e) : 0.f;
  const bool any = __any_sync(0xffffffffu, took);
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = 0.f;
  if (any) {
    float dj = 0.f;  // gradient of slot `lane`'s logit
    if (p.renormalize || p.sigmoid) {
      const float v = p.sigmoid ? log_sigmoid(le) : le;
      if (p.renormalize) {
        const float top = warp_max(took ? v : -INFINITY);
        const float ex = took ? expf(v - top) : 0.f;
        const float w = ex / warp_sum(ex);
        const float mean = warp_sum(took ? g * w : 0.f);
        dj = took ? w * (g - mean) : 0.f;
      } else {
        dj = took ? expf(v) * g : 0.f;
      }
      if (p.sigmoid) dj = took ? dj / (1.f + expf(le)) : 0.f;
    } else {
      float l[V];
      load_row<V, T>(row, e0, p.experts, p.wide != 0, l);
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
      top = warp_max(top);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] = expf(l[i] - top);
      const float inv = 1.f / warp_sum(sum);
      const float pe = took ? expf(le - top) * inv : 0.f;
      const float mean = warp_sum(took ? g * pe : 0.f);
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = -l[i] * inv * mean;
      dj = pe * g;
    }
    for (int j = 0; j < p.topk; ++j) {
      const int ej = __shfl_sync(0xffffffffu, took ? e : -1, j);
      const float x = __shfl_sync(0xffffffffu, dj, j);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ej == e0 + i) d[i] += x;
    }
  }
  T* out = static_cast<T*>(p.dlogits) + t * p.experts;
  constexpr int kBytes = V * int(sizeof(T));
  if (kBytes % 16 == 0 && p.wide) {
    if constexpr (kBytes % 16 == 0) {
      if (e0 < p.experts) {
        uint4 raw[kBytes / 16];
        T* o = reinterpret_cast<T*>(raw);
#pragma unroll
        for (int i = 0; i < V; ++i) store_logit(o + i, d[i]);
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(out + e0)[i] = raw[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < p.experts) store_logit(out + e0 + i, d[i]);
  }
}

// Experts per lane: the least power of two that covers them with 32 lanes.
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

template <class T>
cudaError_t route(const RouteParams& p, bool scored, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value;
    RouteParams q = p;
    q.wide = p.experts % V == 0 && p.ld * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
    auto kern = scored ? route_kernel<V, T, true> : route_kernel<V, T, false>;
    return launch_dependent(kern, unsigned((p.tokens + kWarps - 1) / kWarps), 32 * kWarps, 0, stream, 1, q);
  });
}

template <class T>
cudaError_t route_backward(const RouteBackParams& p, cudaStream_t stream) {
  return by_width(lane_experts(p.experts), [&](auto v) {
    constexpr int V = decltype(v)::value;
    RouteBackParams q = p;
    q.wide = p.experts % V == 0 && p.ld * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
             p.experts * sizeof(T) % 16 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % 16 == 0;
    return launch_dependent(route_backward_kernel<V, T>, unsigned((p.tokens + kWarps - 1) / kWarps), 32 * kWarps, 0,
                            stream, 1, q);
  });
}

int check(const void* logits, int dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t topk, int score) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (tokens < 0 || experts < 1 || experts > GMM_MAX_GROUPS || topk < 1 || topk > experts || topk > GMM_MAX_TOPK ||
      ld < experts || (tokens + kWarps - 1) / kWarps > INT32_MAX)
    return GMM_ERR_SHAPE;
  if (score != GMM_SCORE_SOFTMAX && score != GMM_SCORE_SIGMOID) return GMM_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == GMM_DTYPE_F32 ? 4 : 2) != 0) return GMM_ERR_ALIGN;
  return GMM_OK;
}

bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace
}  // namespace gmmk

extern "C" int gmm_route(const void* logits, int logits_dtype, int64_t tokens, int32_t num_experts, int64_t logits_ld,
                         int32_t topk, int score, int renormalize, float scale, const float* select_bias,
                         const uint8_t* token_mask, float* weights, int32_t* experts, void* stream) {
  using namespace gmmk;
  const bool scored = (score & GMM_SCORE_BIASED) != 0 && select_bias != nullptr;
  score &= ~GMM_SCORE_BIASED;
  if (int st = check(logits, logits_dtype, tokens, num_experts, logits_ld, topk, score)) return st;
  if (tokens > 0 && (logits == nullptr || weights == nullptr || experts == nullptr))
    return GMM_ERR_NULL;
  if (!aligned4(select_bias) || !aligned4(weights) || !aligned4(experts)) return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const RouteParams p{logits, tokens, logits_ld, num_experts, topk, score == GMM_SCORE_SIGMOID, renormalize != 0, 0,
                      scale, select_bias, token_mask, weights, experts};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_dtype == GMM_DTYPE_F32 ? route<float>(p, scored, s) : route<__nv_bfloat16>(p, scored, s);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}

extern "C" int gmm_route_backward(const float* dweights, const int32_t* experts, const void* logits, int logits_dtype,
                                  int64_t tokens, int32_t num_experts, int64_t logits_ld, int32_t topk, int score,
                                  int renormalize, float scale, void* dlogits, void* stream) {
  using namespace gmmk;
  if (int st = check(logits, logits_dtype, tokens, num_experts, logits_ld, topk, score)) return st;
  if (tokens > 0 && (dweights == nullptr || experts == nullptr || logits == nullptr || dlogits == nullptr))
    return GMM_ERR_NULL;
  if (!aligned4(dweights) || !aligned4(experts) ||
      reinterpret_cast<uintptr_t>(dlogits) % (logits_dtype == GMM_DTYPE_F32 ? 4 : 2) != 0)
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const RouteBackParams p{dweights, experts, logits, tokens, logits_ld, num_experts, topk,
                          score == GMM_SCORE_SIGMOID, renormalize != 0, 0, scale, dlogits};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      logits_dtype == GMM_DTYPE_F32 ? route_backward<float>(p, s) : route_backward<__nv_bfloat16>(p, s);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
