// Weights in 4-bit integers: bf16 or f32 rows to codes with a bf16 scale, and a zero
// point, for each group of 32, 64 or 128 values of a row, and back.
//
//   scale = bf16(max|x| / 7),      code = round(x / scale) within -8 .. 7
//   scale = bf16((hi - lo) / 15),  zero = round(-lo / scale),
//                                  code = round(x / scale) + zero within 0 .. 15
//
// Codes are those of exact arithmetic.  An fp32 quotient x / s rounds, but never onto
// a point half way between two whole numbers unless the exact quotient is that point:
// s has 8 significant bits and the half-way point h at most 5, so h s is an fp32 value,
// and an x one unit of 2^-23 off it makes a quotient more than half a unit off h
// (1 / s's significand against 1 / 2).  That leaves room of 2^-32 relative for the
// quotient's own error, and x r + x r', with r the rounded reciprocal of s and r' what
// it lacks, is correct to 2^-40 before its one rounding, at a third of a division's
// instructions.  Scales whose reciprocal is not a normal number are divided by.
//
// Bound by memory: 2 bytes read and 1/2 written per value (bf16).  A warp takes a
// window of 256 values of a row, a lane 8 of them.
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_experts.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWindow = 256, kThreads = 256;

struct QuantParams {
  const void* x;
  int64_t rows, rows_per_batch, ld;  // of all batches
  int64_t k, windows;
  uint8_t* codes;
  __nv_bfloat16* scale;
  uint8_t* zero;
};

template <class T>
__device__ __forceinline__ void load8(const T* p, bool wide, float (&v)[8]) {
  if (wide) {
    uint4 raw[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = float(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = float(p[i]);
  }
}

// round(x / s) of exact quotients.
struct Quotient {
  float s, r, rest;
  bool plain;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale) {
    plain = !(s >= 0x1p-100f && s <= 0x1p100f);
    r = __frcp_rn(s), rest = fmaf(-s, r, 1.f) * r;
  }
  __device__ __forceinline__ float operator()(float x) const {
    return rintf(plain ? __fdiv_rn(x, s) : fmaf(x, r, x * rest));
  }
};

// kLanes lanes hold a group (8 values each).
template <class T, int kLanes, bool kZero>
__global__ void __launch_bounds__(kThreads) quantize_int4_kernel(QuantParams p, bool wide) {
  griddep_begin();
  p.x = after_begin(p.x);
  constexpr int kEach = 32 / kLanes;  // groups of a window
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  if (w >= p.rows * p.windows) return;
  const int64_t row = w / p.windows, window = w - row * p.windows;
  const int64_t c = window * kWindow + lane * 8;
  const bool in = c < p.k;  // k is whole groups, so all of a group's lanes are
  float v[8];
  if (in) {
    load8<T>(static_cast<const T*>(p.x) + row * p.ld + c, wide, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  float span;
  float lo = 0.f;
  bool fine = true;
  if constexpr (kZero) {
    float hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]), fine &= fabsf(v[i]) <= 3.402823466e38f;
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
      fine &= __shfl_xor_sync(0xffffffffu, int(fine), d) != 0;
    }
    span = hi - lo;
    fine &= span <= 3.402823466e38f;
  } else {
    uint32_t top = 0;  // magnitudes as ordered bits: a NaN is above infinity
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    span = __uint_as_float(top);
    fine = top < 0x7F800000u;
  }
  const __nv_bfloat16 scale = __float2bfloat16_rn(fine ? __fdiv_rn(span, kZero ? 15.f : 7.f) : __uint_as_float(0x7FC00000u));
  const float s = __bfloat162float(scale);
  uint32_t code = 0;
  float zero = 0.f;
  if (s > 0.f) {
    const Quotient q(s);
    if constexpr (kZero) zero = fminf(q(-lo), 15.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = kZero ? fminf(fmaxf(q(v[i]) + zero, 0.f), 15.f) : fminf(fmaxf(q(v[i]), -8.f), 7.f);
      code |= (uint32_t(int(n)) & 15u) << (4 * i);
    }
  }
  if (in) *reinterpret_cast<uint32_t*>(p.codes + row * (p.k / 2) + c / 2) = code;
  if (lane % kLanes == 0) {
    const int64_t batch = row / p.rows_per_batch, r = row - batch * p.rows_per_batch;
    const int64_t at = ((batch * p.windows + window) * p.rows_per_batch + r) * kEach + lane / kLanes;
    p.scale[at] = in ? scale : __float2bfloat16_rn(0.f);
    if constexpr (kZero) p.zero[at] = in ? uint8_t(zero) : 0;
  }
}

struct DequantParams {
  const uint8_t* codes;
  const __nv_bfloat16* scale;
  const uint8_t* zero;
  int64_t rows, rows_per_batch, k, windows;
  void* out;
};

template <class T, int kLanes>
__global__ void __launch_bounds__(kThreads) dequantize_int4_kernel(DequantParams p, bool wide) {
  griddep_begin();
  p.codes = after_begin(p.codes), p.scale = after_begin(p.scale), p.zero = after_begin(p.zero);
  constexpr int kEach = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  if (w >= p.rows * p.windows) return;
  const int64_t row = w / p.windows, window = w - row * p.windows;
  const int64_t c = window * kWindow + lane * 8;
  if (c >= p.k) return;
  const int64_t batch = row / p.rows_per_batch, r = row - batch * p.rows_per_batch;
  const int64_t at = ((batch * p.windows + window) * p.rows_per_batch + r) * kEach + lane / kLanes;
  const uint32_t code = __ldg(reinterpret_cast<const uint32_t*>(p.codes + row * (p.k / 2) + c / 2));
  const float s = __bfloat162float(p.scale[at]);
  const int zero = p.zero != nullptr ? p.zero[at] : 8;
  const uint32_t flip = p.zero != nullptr ? 0u : 8u;  // two's complement + 8
  T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = T(s * float(int(((code >> (4 * i)) & 15u) ^ flip) - zero));
  T* out = static_cast<T*>(p.out) + row * p.k + c;
  if (wide) {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(out)[i] = reinterpret_cast<const uint4*>(v)[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = v[i];
  }
}

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

template <class F>
cudaError_t by_group(int group, F&& go) {
  switch (group) {
    case 32: return go(std::integral_constant<int, 4>{});
    case 64: return go(std::integral_constant<int, 8>{});
    default: return go(std::integral_constant<int, 16>{});
  }
}

int check(int dtype, int32_t batch, int64_t rows, int64_t k, int64_t ld, int32_t group) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (batch < 0 || rows < 0 || k < 1 || k > kMaxSize || rows > kMaxSize || ld < k ||
      (group != 32 && group != 64 && group != 128) || k % group != 0)
    return GMM_ERR_SHAPE;
  const int64_t all = int64_t(batch) * rows;
  if (all > kMaxSize * 8 || (all > 0 && (k + kWindow - 1) / kWindow > kMaxSize * 8 / all)) return GMM_ERR_SHAPE;
  return GMM_OK;
}

unsigned blocks_of(int64_t warps) { return unsigned((warps * 32 + kThreads - 1) / kThreads); }

}  // namespace
}  // namespace gmmk

extern "C" int gmm_quantize_int4(const void* x, int x_dtype, int32_t batch, int64_t rows_per_batch, int64_t k,
                                 int64_t x_ld, int32_t group, void* codes, void* scale, void* zero, void* stream) {
  using namespace gmmk;
  if (int st = check(x_dtype, batch, rows_per_batch, k, x_ld, group)) return st;
  const int64_t rows = int64_t(batch) * rows_per_batch;
  if (rows > 0 && (x == nullptr || codes == nullptr || scale == nullptr)) return GMM_ERR_NULL;
  const int size = x_dtype == GMM_DTYPE_F32 ? 4 : 2;
  if (misaligned(x, size) || misaligned(codes, 16) || misaligned(scale, 16) || misaligned(zero, 4))
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (rows == 0) return GMM_OK;
  const QuantParams p{x, rows, rows_per_batch, x_ld, k, (k + kWindow - 1) / kWindow, static_cast<uint8_t*>(codes),
                      static_cast<__nv_bfloat16*>(scale), static_cast<uint8_t*>(zero)};
  const bool wide = !misaligned(x, 16) && x_ld * size % 16 == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = blocks_of(rows * p.windows);
  const cudaError_t e = by_group(group, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto kern = x_dtype == GMM_DTYPE_F32
                    ? (zero != nullptr ? quantize_int4_kernel<float, L, true> : quantize_int4_kernel<float, L, false>)
                    : (zero != nullptr ? quantize_int4_kernel<__nv_bfloat16, L, true>
                                       : quantize_int4_kernel<__nv_bfloat16, L, false>);
    return launch_dependent(kern, grid, kThreads, 0, s, 1, p, wide);
  });
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}

extern "C" int gmm_dequantize_int4(const void* codes, const void* scale, const void* zero, int32_t group, int32_t batch,
                                   int64_t rows_per_batch, int64_t k, void* out, int out_dtype, void* stream) {
  using namespace gmmk;
  if (int st = check(out_dtype, batch, rows_per_batch, k, k, group)) return st;
  const int64_t rows = int64_t(batch) * rows_per_batch;
  if (rows > 0 && (codes == nullptr || scale == nullptr || out == nullptr)) return GMM_ERR_NULL;
  const int size = out_dtype == GMM_DTYPE_F32 ? 4 : 2;
  if (misaligned(codes, 4) || misaligned(scale, 2) || misaligned(out, size)) return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (rows == 0) return GMM_OK;
  const DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const __nv_bfloat16*>(scale),
                        static_cast<const uint8_t*>(zero), rows, rows_per_batch, k, (k + kWindow - 1) / kWindow, out};
  const bool wide = !misaligned(out, 16);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = blocks_of(rows * p.windows);
  const cudaError_t e = by_group(group, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto kern = out_dtype == GMM_DTYPE_F32 ? dequantize_int4_kernel<float, L> : dequantize_int4_kernel<__nv_bfloat16, L>;
    return launch_dependent(kern, grid, kThreads, 0, s, 1, p, wide);
  });
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
