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
// Bound by memory, 2 bytes read and 1/2 written per value (bf16), and nearly by the instructions that
// a value takes, so these are few: a lane takes 16 consecutive values, a warp 512 of a row at a time;
// codes are rounded by adding 1.5 2^23 and put together as they stand, sum of 16^i (1.5 2^23 + code),
// the constant part taken off at the end.  Without zero points nothing has to be kept within -8 .. 7,
// because a scale of 8 bits is at most 2^-8 of itself below max|x| / 7 (subnormal ones take a longer way).
// Measured: 8 x 4096 x 4096, groups of 128: from bf16 58 us (338 MB, 5.8 TB/s), with zero points 70; from f32 90 (6.7)
// and 94; back to bf16 51.8 (6.5) and 52.2, to f32 130 (4.7) and 120.  2048 x 4000 f32, groups of 32 with zero
// points, 8.6 and back to bf16 5.2: one wave of 4096 warps with four turns each.
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
  int64_t rows, ld;  // of all batches
  int32_t rows_per_batch, parts_log2;  // warps to a row
  int32_t k, windows, wide;
  uint8_t* codes;
  __nv_bfloat16* scale;
  uint8_t* zero;
};

// 16 values as they are stored.
template <class T>
struct Values {
  static constexpr int kWords = 16 * int(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zeros() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = uint32_t(__ldg(h + 2 * i)) | uint32_t(__ldg(h + 2 * i + 1)) << 16;
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // The largest magnitude as ordered bits: a NaN is above infinity.
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      return max(m & 0xFFFFu, m >> 16) << 16;
    }
  }
};

// Two fp32 operations at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 w, x, y, z; "
      "mov.b64 {%0, %1}, w;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

constexpr float kRound = 12582912.f;                  // 1.5 2^23: a sum with it is rounded to a whole number
constexpr uint32_t kRoundBits = 0x4B400000u;
constexpr float kLargest = 3.402823466e38f;

// kLanes lanes hold a group (16 values each).
template <class T, int kLanes, bool kZero>
__global__ void __launch_bounds__(kThreads) quantize_int4_kernel(QuantParams p) {
  griddep_begin();
  p.x = after_begin(p.x);
  constexpr int kEach = 16 / kLanes;  // groups of a window
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t row = warp >> p.parts_log2;
  if (row >= p.rows) return;
  const int part = int(warp) & ((1 << p.parts_log2) - 1), step = 512 << p.parts_log2;
  const int batch = int(row) / p.rows_per_batch, r = int(row) - batch * p.rows_per_batch;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  uint8_t* codes = p.codes + row * (p.k / 2);
  const int64_t at_batch = int64_t(batch) * p.windows;
  const int64_t whole = int64_t(p.windows) * kWindow;
  // k is whole groups, so all of a group's lanes are within it or none
  auto read = [&](int64_t c) {
    Values<T> v;
    if (c < p.k)
      v.load(x + c, p.wide != 0);
    else
      v.zeros();
    return v;
  };
  Values<T> next = read(part * 512 + lane * 16);
#pragma unroll 1
  for (int64_t c = part * 512 + lane * 16; c - lane * 16 < whole; c += step) {
    const bool in = c < p.k;
    const Values<T> v = next;
    next = read(c + step);  // on its way while these are encoded
    float span, lo = 0.f;
    bool fine = true;
    if constexpr (kZero) {
      float hi = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
      fine = v.top() < 0x7F800000u;
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        fine &= __shfl_xor_sync(0xffffffffu, int(fine), d) != 0;
      }
      span = hi - lo;
      fine &= span <= kLargest;
    } else {
      uint32_t top = v.top();
#pragma unroll
      for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      span = __uint_as_float(top);
      fine = top < 0x7F800000u;
    }
    const __nv_bfloat16 scale =
        __float2bfloat16_rn(fine ? __fdiv_rn(span, kZero ? 15.f : 7.f) : __uint_as_float(0x7FC00000u));
    const float s = __bfloat162float(scale);
    uint32_t code[2] = {0, 0};
    float zero = 0.f;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
      const float r = __frcp_rn(s), rest = fmaf(-s, r, 1.f) * r;
      float most = 0.f;
      if constexpr (kZero) zero = fminf(rintf(fmaf(-lo, r, -lo * rest)), 15.f), most = 15.f - zero;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t sum = 0;
#pragma unroll
        for (int i = 6; i >= 0; i -= 2) {
          const float2 a = make_float2(v[8 * h + i], v[8 * h + i + 1]);
          float2 q = fma2(a, make_float2(r, r), mul2(a, make_float2(rest, rest)));
          if constexpr (kZero) q.x = fminf(q.x, most), q.y = fminf(q.y, most);
          q = add2(q, make_float2(kRound, kRound));
          sum = (sum * 16 + __float_as_uint(q.y)) * 16 + __float_as_uint(q.x);
        }
        sum -= kRoundBits * 0x11111111u;  // sum of 16^i code, which borrows where codes are negative
        code[h] = kZero ? sum + uint32_t(int(zero)) * 0x11111111u : (sum + 0x88888888u) ^ 0x88888888u;
      }
    } else if (s > 0.f) {  // reciprocals that are no normal numbers
      if constexpr (kZero) zero = fminf(rintf(__fdiv_rn(-lo, s)), 15.f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float q = rintf(__fdiv_rn(v[i], s));
        const float n = kZero ? fminf(fmaxf(q + zero, 0.f), 15.f) : fminf(fmaxf(q, -8.f), 7.f);
        code[i / 8] |= (uint32_t(int(n)) & 15u) << (4 * (i % 8));
      }
    }
    if (in) *reinterpret_cast<uint2*>(codes + c / 2) = make_uint2(code[0], code[1]);
    const int64_t window = c / kWindow;
    if (lane % kLanes == 0 && window < p.windows) {
      const int64_t at = ((at_batch + window) * p.rows_per_batch + r) * kEach + lane % 16 / kLanes;
      p.scale[at] = in ? scale : __float2bfloat16_rn(0.f);
      if constexpr (kZero) p.zero[at] = in ? uint8_t(zero) : 0;
    }
  }
}

struct DequantParams {
  const uint8_t* codes;
  const __nv_bfloat16* scale;
  const uint8_t* zero;
  int64_t rows;
  int32_t rows_per_batch, parts_log2, k, windows, wide;
  void* out;
};

// A warp takes windows of a row, a lane 8 codes, kLanes lanes a group.
template <class T, int kLanes, bool kZero>
__global__ void __launch_bounds__(kThreads) dequantize_int4_kernel(DequantParams p) {
  griddep_begin();
  p.codes = after_begin(p.codes), p.scale = after_begin(p.scale), p.zero = after_begin(p.zero);
  constexpr int kEach = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t row = warp >> p.parts_log2;
  if (row >= p.rows) return;
  const int part = int(warp) & ((1 << p.parts_log2) - 1), step = 1 << p.parts_log2;
  const int batch = int(row) / p.rows_per_batch, r = int(row) - batch * p.rows_per_batch;
  const uint8_t* codes = p.codes + row * (p.k / 2) + lane * 4;
  T* out = static_cast<T*>(p.out) + row * p.k + lane * 8;
  const int64_t first = (int64_t(batch) * p.windows * p.rows_per_batch + r) * kEach + lane / kLanes;
  const int64_t pitch = int64_t(p.rows_per_batch) * kEach;
  // four windows on their way
  constexpr int kAhead = 4;
  for (int64_t w0 = part; w0 < p.windows; w0 += kAhead * step) {
    uint32_t words[kAhead], zeros[kAhead];
    __nv_bfloat16 scales[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t w = w0 + i * step;
      if (w * kWindow + lane * 8 < p.k) {
        words[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + w * (kWindow / 2)));
        scales[i] = __ldg(p.scale + first + w * pitch);
        if constexpr (kZero) zeros[i] = __ldg(p.zero + first + w * pitch);
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int64_t w = w0 + a * step;
      if (w * kWindow + lane * 8 >= p.k) break;
      const uint32_t code = words[a];
      const __nv_bfloat16 s = scales[a];
      // a nibble or-ed into 128 is 128 + code (two's complement + 8 is its top bit flipped); 128 + zero off it
      uint32_t off = 0x43084308u;
      if constexpr (kZero) off = 0x43004300u + zeros[a] * 0x00010001u;
      uint32_t n[4];  // codes 0 and 4, 1 and 5, 2 and 6, 3 and 7
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t raw = (code >> (4 * i) & 0x000F000Fu) ^ (kZero ? 0x43004300u : 0x43084308u);
        const __nv_bfloat162 v =
            __hsub2(reinterpret_cast<const __nv_bfloat162&>(raw), reinterpret_cast<const __nv_bfloat162&>(off));
        n[i] = reinterpret_cast<const uint32_t&>(v);
      }
      T* to = out + w * kWindow;
      if constexpr (sizeof(T) == 2) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // products of 4 and 8 bits, rounded once
          const uint32_t pair = __byte_perm(n[i % 2 * 2], n[i % 2 * 2 + 1], i < 2 ? 0x5410 : 0x7632);
          const __nv_bfloat162 y = __hmul2(reinterpret_cast<const __nv_bfloat162&>(pair), __nv_bfloat162(s, s));
          v[i] = reinterpret_cast<const uint32_t&>(y);
        }
        if (p.wide) {
          *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) reinterpret_cast<uint16_t*>(to)[i] = uint16_t(v[i / 2] >> (16 * (i % 2)));
        }
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = __bfloat162float(s) * __uint_as_float(n[i] << 16);
          v[i + 4] = __bfloat162float(s) * __uint_as_float(n[i] & 0xFFFF0000u);
        }
        if (p.wide) {
          reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) to[i] = v[i];
        }
      }
    }
  }
}

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

int check(int dtype, int32_t batch, int64_t rows, int64_t k, int64_t ld, int32_t group) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (batch < 0 || rows < 0 || k < 1 || k > kMaxSize || rows > kMaxSize || ld < k ||
      (group != 32 && group != 64 && group != 128) || k % group != 0 || int64_t(batch) * rows > kMaxSize)
    return GMM_ERR_SHAPE;
  return GMM_OK;
}

// Warps to a row: as few as keep some 4000 on the GPU, at most one for each `each` values (one row of 16384
// 1.5 us, with one warp 12; 256 rows of 4096 2.2 and 4.4).
int parts_of(int64_t rows, int64_t k, int64_t each) {
  int lg = 0;
  while (lg < 20 && (rows << lg) < 4096 && (each << lg) < k) ++lg;
  return lg;
}
unsigned blocks_of(int64_t rows, int lg) { return unsigned(((rows << lg) * 32 + kThreads - 1) / kThreads); }

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
  const int lg = parts_of(rows, k, 512);
  const QuantParams p{x, rows, x_ld, int32_t(rows_per_batch), lg, int32_t(k), int32_t((k + kWindow - 1) / kWindow),
                      !misaligned(x, 16) && x_ld * size % 16 == 0, static_cast<uint8_t*>(codes),
                      static_cast<__nv_bfloat16*>(scale), static_cast<uint8_t*>(zero)};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto kern = x_dtype == GMM_DTYPE_F32
                    ? (zero != nullptr ? quantize_int4_kernel<float, L, true> : quantize_int4_kernel<float, L, false>)
                    : (zero != nullptr ? quantize_int4_kernel<__nv_bfloat16, L, true>
                                       : quantize_int4_kernel<__nv_bfloat16, L, false>);
    return launch_dependent(kern, blocks_of(rows, lg), kThreads, 0, s, 1, p);
  };
  const cudaError_t e = group == 32   ? go(std::integral_constant<int, 2>{})
                        : group == 64 ? go(std::integral_constant<int, 4>{})
                                      : go(std::integral_constant<int, 8>{});
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
  const int lg = parts_of(rows, k, kWindow);
  const DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const __nv_bfloat16*>(scale),
                        static_cast<const uint8_t*>(zero), rows, int32_t(rows_per_batch), lg, int32_t(k),
                        int32_t((k + kWindow - 1) / kWindow), !misaligned(out, 16), out};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto kern = out_dtype == GMM_DTYPE_F32
                    ? (zero != nullptr ? dequantize_int4_kernel<float, L, true> : dequantize_int4_kernel<float, L, false>)
                    : (zero != nullptr ? dequantize_int4_kernel<__nv_bfloat16, L, true>
                                       : dequantize_int4_kernel<__nv_bfloat16, L, false>);
    return launch_dependent(kern, blocks_of(rows, lg), kThreads, 0, s, 1, p);
  };
  const cudaError_t e = group == 32   ? go(std::integral_constant<int, 4>{})
                        : group == 64 ? go(std::integral_constant<int, 8>{})
                                      : go(std::integral_constant<int, 16>{});
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
