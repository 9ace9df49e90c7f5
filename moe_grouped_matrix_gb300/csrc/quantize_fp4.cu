// Microscaled 4-bit floating point: bf16 or f32 rows to e2m1 codes with a scale
// for every block of a row, and back.
//
//   NVFP4  16 codes a block, e4m3 block scales, a power of two per row that puts
//          the row's largest value at the top of the block scales' range;
//   MXFP4  32 codes a block, E8M0 block scales.
//
// A power of two per row costs no accuracy (block scales keep 3 bits wherever in
// e4m3's normal range they lie) and keeps every quotient exact to decide: x and
// the block maximum scale without rounding, and the nearest code depends on a
// quotient of two short significands.  An fp32 quotient rounds, but never onto
// or across a point half way between two codes (or two e4m3 values) unless the
// exact quotient is that point: with a numerator one unit of 2^-23 off the half-
// way product the quotient is more than half a unit off the half-way point,
// because the point's significand is over half of the numerator's.  So codes and
// scales are those of exact arithmetic.  x / s is taken as x r + x r', with r the
// rounded reciprocal of s and r' what it lacks: correct to 2^-40 before its one
// rounding (r alone is wrong on the half-way points of s = 15 2^j), at a third
// of a division's instructions.
//
// Bound by memory: 2 bytes read and 9/16 written per value (17/32 for MXFP4).
// A row is read once: a warp or a CTA holds it in registers (rows of over 16384
// values are read twice).  16384 rows of 4096 in bf16: MXFP4
// 27 us, NVFP4 31 us, of which about 4 are a launch's; the bytes take 25.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kMaxThreads = 256;

struct QuantParams {
  const void* x;
  int64_t rows_per_batch, k, ld;
  int64_t in_rows;       // batch * rows_per_batch
  const int32_t* rows;   // NULL, or the order's rows [tokens, topk]
  const int32_t* source;
  int32_t topk;
  uint8_t* codes;
  uint8_t* scale;
  float* row_scale;
};

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // -126..127

// The least e with a <= 2^(e + shift) * (1 + limit 2^-23), for finite a > 0.
__device__ __forceinline__ int least_exponent(uint32_t bits, uint32_t limit, int shift) {
  if (bits < 0x00800000u) {  // subnormal
    bits = __float_as_uint(__uint_as_float(bits) * 0x1p64f);
    shift += 64;
  }
  return int(bits >> 23) - 127 - shift + ((bits & 0x7FFFFFu) > limit ? 1 : 0);
}

// What a thread holds of a row: 16 values as stored.
template <class T>
struct Unit {
  static constexpr int kWords = 16 * int(sizeof(T)) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
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
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__ldg(reinterpret_cast<const float*>(p) + i));
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = uint32_t(__ldg(h + 2 * i)) | uint32_t(__ldg(h + 2 * i + 1)) << 16;
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  // The largest magnitude as fp32 bits: kInfBits or more when a value is not finite.
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t a = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) a = max(a, w[i] & 0x7FFFFFFFu);
      return a;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a = __vmaxu2(a, w[i] & 0x7FFF7FFFu);
      return max(a & 0xFFFFu, a >> 16) << 16;
    }
  }
  // The signs, each at its code's top bit: the codes of zeros.
  __device__ __forceinline__ uint2 signs() const {
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i / 8] |= (__float_as_uint(value(i)) >> 31) << (4 * (i % 8) + 3);
    return make_uint2(out[0], out[1]);
  }
  // Codes of value * up / s, s > 0 with 4 significant bits.
  __device__ __forceinline__ uint2 encode(float up, float s) const {
    const float r = __frcp_rn(s), rest = fmaf(-s, r, 1.f) * r;
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = value(8 * h + i) * up;
        q[i] = fmaf(y, r, y * rest);
      }
      out[h] = pack(q);
    }
    return make_uint2(out[0], out[1]);
  }
  // Codes of value * f.
  __device__ __forceinline__ uint2 encode(float f) const {
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = value(8 * h + i) * f;
      out[h] = pack(q);
    }
    return make_uint2(out[0], out[1]);
  }
  static __device__ __forceinline__ uint32_t pack(const float (&q)[8]) {
    uint32_t out;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return out;
  }
};
constexpr uint32_t kInfBits = 0x7F800000u;

// e4m3's value of a byte below 0x7F.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  // 3 bits after the point, exponent bias 7, subnormals below 2^-6
  return byte >= 8 ? __uint_as_float((byte << 20) + (120u << 23)) : float(byte) * 0x1p-9f;
}

// kThreads threads quantise one input row and write it to its rows of the
// result; thread i holds units i, i + kThreads, .. of 16 values.  A unit is a
// block of NVFP4, or half a block of MXFP4, whose other half the next lane has.
// kUnits > 0: a thread's units, all in registers; 0: any number, read again
// for the codes.
template <class T, bool kNv, int kThreads, int kUnits, bool kOrder>
__global__ void __launch_bounds__(kThreads == 32 ? 128 : kThreads) quantize_fp4_kernel(QuantParams p, bool wide) {
  griddep_begin();
  p.x = after_begin(p.x), p.rows = after_begin(p.rows), p.source = after_begin(p.source);
  constexpr int kRows = kThreads == 32 ? 4 : 1;  // rows a CTA
  __shared__ uint32_t warp_max[kThreads / 32];
  const int lane = threadIdx.x & 31;
  const int tid = kRows > 1 ? lane : int(threadIdx.x);
  const int64_t row = int64_t(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x >> 5 : 0);
  if (kRows > 1 && row >= p.in_rows) return;
  const T* x = static_cast<const T*>(p.x) + row * p.ld;
  const int32_t units = int32_t(p.k / 16);
  constexpr int32_t kWindow = kNv ? 16 : 32;  // units of a window
  const int32_t windows = (units + kWindow - 1) / kWindow, padded = windows * kWindow;
  constexpr int kHeld = kUnits > 0 ? kUnits : 1;
  Unit<T> held[kHeld];
  uint32_t high = 0;
  if constexpr (kUnits > 0) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int32_t u = i * kThreads + tid;
      if (u < units)
        held[i].load(x + 16 * int64_t(u), wide);
      else
        held[i].zero();
    }
    if constexpr (kNv) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const uint32_t a = held[i].amax();
        if (a < kInfBits) high = max(high, a);
      }
    }
  } else if constexpr (kNv) {
    for (int32_t u = tid; u < units; u += kThreads) {
      held[0].load(x + 16 * int64_t(u), wide);
      const uint32_t a = held[0].amax();
      if (a < kInfBits) high = max(high, a);
    }
  }
  float row_scale = 1.f, up = 1.f;
  if constexpr (kNv) {
    high = __reduce_max_sync(0xffffffffu, high);
    if constexpr (kThreads > 32) {
      if (lane == 0) warp_max[threadIdx.x >> 5] = high;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) high = max(high, warp_max[w]);
    }
    if (high != 0) {
      const int e = max(least_exponent(high, 0x280000u, 11), -126);  // 6 * 448 = 1.3125 * 2^11
      row_scale = exp2_int(e), up = exp2_int(-e);
    }
  }
  // where the row goes, and which rows past the groups this one's slots clear
  const int64_t batch = kOrder ? 0 : row / p.rows_per_batch;
  const int64_t out_rows = kOrder ? p.rows_per_batch * p.topk : p.rows_per_batch;
  int32_t to = int32_t(row - batch * p.rows_per_batch), none = -1;
  if constexpr (kOrder) {
    to = -1;
    if (lane < p.topk) {
      to = __ldg(p.rows + row * p.topk + lane);
      to = to < out_rows ? to : -1;
      none = __ldg(p.source + row * p.topk + lane) < 0 ? int32_t(row * p.topk + lane) : -1;
    }
  }
  uint8_t* scale = p.scale + batch * windows * out_rows * 16;
  uint8_t* codes = p.codes + batch * out_rows * (p.k / 2);
  auto store = [&](int32_t u, int64_t r, uint2 c, uint32_t byte) {
    if (u < units) *reinterpret_cast<uint2*>(codes + r * (p.k / 2) + 8 * int64_t(u)) = c;
    const int32_t b = kNv ? u : u / 2;  // the block
    if (u < padded && (kNv || (u & 1) == 0)) scale[(int64_t(b / 16) * out_rows + r) * 16 + b % 16] = uint8_t(byte);
  };
  const int32_t steps = kUnits > 0 ? kUnits : (padded + kThreads - 1) / kThreads;
#pragma unroll
  for (int32_t i = 0; i < steps; ++i) {
    const int32_t u = i * kThreads + tid;
    if constexpr (kUnits == 0) {
      if (u < units)
        held[0].load(x + 16 * int64_t(u), wide);
      else
        held[0].zero();
    }
    const Unit<T>& v = held[kUnits > 0 ? i : 0];
    uint32_t a = v.amax(), byte;
    uint2 c = make_uint2(0u, 0u);
    if constexpr (kNv) {
      if (a >= kInfBits) {
        byte = 0x7Fu;
      } else {
        const float q = __fdiv_rn(__uint_as_float(a) * up, 6.f);
        uint16_t e8;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.f), "f"(q));
        byte = e8 & 0xFFu;
        c = byte != 0 ? v.encode(up, e4m3_value(byte)) : v.signs();
      }
    } else {
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      if (a >= kInfBits) {
        byte = 255u;
      } else if (a == 0) {
        byte = 0u;
        c = v.signs();
      } else {
        const int e = max(least_exponent(a, 0x400000u, 2), -127);  // 6 = 1.5 * 2^2
        byte = uint32_t(e + 127);
        c = v.encode(exp2_int(-e));  // e <= 126
      }
    }
    if (u >= units) byte = 0u;
    if constexpr (kOrder) {
      for (int j = 0; j < p.topk; ++j) {
        const int32_t r = __shfl_sync(0xffffffffu, to, j), z = __shfl_sync(0xffffffffu, none, j);
        if (r >= 0) store(u, r, c, byte);
        if (z >= 0) store(u, z, make_uint2(0u, 0u), 0u);
      }
    } else {
      store(u, to, c, byte);
    }
  }
  if constexpr (kNv) {
    if (kOrder ? tid < p.topk : tid == 0) {
      if (to >= 0) p.row_scale[batch * out_rows + to] = row_scale;
      if (none >= 0) p.row_scale[none] = 1.f;
    }
  }
}

struct DequantParams {
  const uint8_t* codes;
  const uint8_t* scale;
  const float* row_scale;
  int64_t rows_per_batch, k;
  void* out;
};

// Two e2m1 codes (a byte, the even one low) as two fp32 values: they are fp16 values.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 t, u, v, w;\n\tmov.b32 {t, u, v, w}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
  __half2 q;
  memcpy(&q, &h, 4);
  return __half22float2(q);
}

// The value of a scale byte.
template <bool kNv>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (kNv) {
    if ((byte & 0x7Fu) == 0x7Fu) return __uint_as_float(0x7FC00000u);
    return byte & 0x80u ? -e4m3_value(byte & 0x7Fu) : e4m3_value(byte);
  } else {
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return byte == 0 ? 0x1p-127f : __uint_as_float(byte << 23);
  }
}

// f = fl32(x * y) on a point half way between two bf16 values, where a second rounding would tie: a unit
// towards the exact product, if it is not that point.
__device__ __noinline__ float off_half_way(float f, float x, float y) {
  const double left = double(x) * double(y) - double(f);  // exact
  if (left == 0.0) return f;
  return __uint_as_float(__float_as_uint(f) + ((left > 0.0) == (f > 0.f) ? 1 : -1));
}

// A CTA for each row; a thread writes 16 bytes at a time (8 bf16 or 4 f32 values), so that a warp's
// store is whole lines, and has four such pieces on their way.
template <class T, bool kNv>
__global__ void __launch_bounds__(kMaxThreads) dequantize_fp4_kernel(DequantParams p) {
  griddep_begin();
  p.codes = after_begin(p.codes), p.scale = after_begin(p.scale), p.row_scale = after_begin(p.row_scale);
  constexpr int kVals = 16 / int(sizeof(T)), kAtOnce = 4;
  constexpr int kBlockPieces = (kNv ? 16 : 32) / kVals;
  const int32_t pieces = int32_t(p.k / kVals);
  const int64_t row = blockIdx.x;
  const int64_t batch = row / p.rows_per_batch, r = row - batch * p.rows_per_batch;
  const int64_t windows = (p.k + (kNv ? 255 : 511)) / (kNv ? 256 : 512);
  const uint8_t* scale = p.scale + (batch * windows * p.rows_per_batch + r) * 16;
  const uint8_t* codes = p.codes + row * (p.k / 2);
  const float rs = kNv ? __ldg(p.row_scale + row) : 1.f;
  uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * p.k);
  for (int32_t u0 = threadIdx.x; u0 < pieces; u0 += kAtOnce * blockDim.x) {
    uint32_t byte[kAtOnce], c[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int32_t u = u0 + i * int32_t(blockDim.x);
      if (u < pieces) {
        const int32_t b = u / kBlockPieces;
        byte[i] = __ldg(scale + int64_t(b / 16) * p.rows_per_batch * 16 + b % 16);
        c[i] = kVals == 8 ? __ldg(reinterpret_cast<const uint32_t*>(codes) + u)
                          : uint32_t(__ldg(reinterpret_cast<const uint16_t*>(codes) + u));
      }
    }
    auto put = [&](auto exact) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int32_t u = u0 + i * int32_t(blockDim.x);
        if (u >= pieces) continue;
        const float s = scale_value<kNv>(byte[i]);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < kVals / 2; ++j) {
          const float2 q = e2m1x2_values(c[i] >> (8 * j));
          float x = q.x * s * rs, y = q.y * s * rs;  // q * s is exact
          if constexpr (sizeof(T) == 4) {
            w[2 * j] = __float_as_uint(x), w[2 * j + 1] = __float_as_uint(y);
          } else {
            if constexpr (!decltype(exact)::value) {
              if ((__float_as_uint(x) & 0xFFFFu) == 0x8000u) x = off_half_way(x, q.x * s, rs);
              if ((__float_as_uint(y) & 0xFFFFu) == 0x8000u) y = off_half_way(y, q.y * s, rs);
            }
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            memcpy(&w[j], &h, 4);
          }
        }
        out[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    // A code times its scale has 6 bits: with a power of two for the row, as gmm_quantize_fp4 gives, the
    // product is exact wherever its bf16 value is not 0.
    if (kNv && sizeof(T) == 2 && (__float_as_uint(rs) & 0x7FFFFFu) != 0)
      put(std::false_type{});
    else
      put(std::true_type{});
  }
}

template <class T, bool kNv, int kThreads, int kUnits>
cudaError_t quantize_as(const QuantParams& p, bool wide, cudaStream_t s) {
  const int64_t blocks = kThreads == 32 ? (p.in_rows + 3) / 4 : p.in_rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  constexpr int kBlock = kThreads == 32 ? 128 : kThreads;
  auto kern = p.rows != nullptr ? quantize_fp4_kernel<T, kNv, kThreads, kUnits, true>
                                : quantize_fp4_kernel<T, kNv, kThreads, kUnits, false>;
  return launch_dependent(kern, unsigned(blocks), kBlock, 0, s, 1, p, wide);
}

// Threads a row and units a thread that cover a row's whole windows.  With many rows a thread takes
// 4 units, so that a row of up to 2048 values is one warp's, with no barrier, and one of 4096 two
// warps' (16384 rows of 4096 bf16 to NVFP4: 28.7 us, one unit a thread 38.9 us); with few rows one unit
// a thread, for the latency (4096 rows of 2048 in expert order, 4 rows each: 8.3 us, 4 units 10.6 us).
// The two meet at some 5000 rows of 1536 or 2048 values, at 10000 of them in expert order, and at 3000 rows
// of 4096: 8192 lies among these (12288 rows of 2048 in expert order 22.0 us, as few 22.3; 6144 rows of
// 2048 8.6 us, as many 8.1; of 4096 15.7, as many 12.6, which it gives away).
template <class T, bool kNv>
cudaError_t quantize(const QuantParams& p, cudaStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ld * sizeof(T) % 16 == 0;
  constexpr int64_t kWindow = kNv ? 16 : 32;
  const int64_t padded = (p.k / 16 + kWindow - 1) / kWindow * kWindow;
  if (padded <= 32) return quantize_as<T, kNv, 32, 1>(p, wide, s);
  if (padded <= 64) return quantize_as<T, kNv, 32, 2>(p, wide, s);
  const bool many = p.in_rows >= 8192;
  if (padded <= 128 && many) return quantize_as<T, kNv, 32, 4>(p, wide, s);
  if (padded <= 128) return quantize_as<T, kNv, 128, 1>(p, wide, s);
  if (padded <= 256 && many) return quantize_as<T, kNv, 64, 4>(p, wide, s);
  if (padded <= 256) return quantize_as<T, kNv, 256, 1>(p, wide, s);
  if (padded <= 512) return quantize_as<T, kNv, 256, 2>(p, wide, s);
  if (padded <= 1024) return quantize_as<T, kNv, 256, 4>(p, wide, s);
  return quantize_as<T, kNv, 256, 0>(p, wide, s);
}

uint64_t address(const void* p) { return uint64_t(reinterpret_cast<uintptr_t>(p)); }

}  // namespace
}  // namespace gmmk

extern "C" int gmm_quantize_fp4(const void* x, int x_dtype, int32_t batch, int64_t rows_per_batch, int64_t k,
                                int64_t x_ld, int format, const int32_t* rows, const int32_t* source, int32_t topk,
                                void* codes, void* block_scale, float* row_scale, void* stream) {
  using namespace gmmk;
  if (format != GMM_FP4_NVFP4 && format != GMM_FP4_MXFP4) return GMM_ERR_DTYPE;
  const bool nv = format == GMM_FP4_NVFP4;
  if (rows_per_batch > 0 && (x == nullptr || codes == nullptr || block_scale == nullptr ||
                             (nv && row_scale == nullptr) || (rows == nullptr) != (source == nullptr)))
    return GMM_ERR_NULL;
  if (x_dtype != GMM_DTYPE_BF16 && x_dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  const bool f32 = x_dtype == GMM_DTYPE_F32;
  if (batch < 1 || rows_per_batch < 0 || rows_per_batch > INT32_MAX || k < 32 || k % 32 != 0 || k > INT32_MAX ||
      x_ld < k)
    return GMM_ERR_SHAPE;
  if (rows == nullptr ? topk != 1 && rows_per_batch > 0
                      : batch != 1 || topk < 1 || topk > GMM_MAX_TOPK || rows_per_batch > INT32_MAX / topk)
    return GMM_ERR_SHAPE;
  if ((address(codes) | address(block_scale)) % 16 != 0 || address(x) % (f32 ? 4 : 2) != 0 ||
      (address(rows) | address(source) | address(row_scale)) % 4 != 0)
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (rows_per_batch == 0) return GMM_OK;
  const QuantParams p{x, rows_per_batch, k, x_ld, int64_t(batch) * rows_per_batch, rows, source, topk,
                      static_cast<uint8_t*>(codes), static_cast<uint8_t*>(block_scale), row_scale};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = f32 ? (nv ? quantize<float, true>(p, s) : quantize<float, false>(p, s))
                            : (nv ? quantize<__nv_bfloat16, true>(p, s) : quantize<__nv_bfloat16, false>(p, s));
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}

extern "C" int gmm_dequantize_fp4(const void* codes, const void* block_scale, const float* row_scale, int format,
                                  int32_t batch, int64_t rows_per_batch, int64_t k, void* out, int out_dtype,
                                  void* stream) {
  using namespace gmmk;
  if (format != GMM_FP4_NVFP4 && format != GMM_FP4_MXFP4) return GMM_ERR_DTYPE;
  const bool nv = format == GMM_FP4_NVFP4;
  if (rows_per_batch > 0 &&
      (codes == nullptr || block_scale == nullptr || out == nullptr || (nv && row_scale == nullptr)))
    return GMM_ERR_NULL;
  if (out_dtype != GMM_DTYPE_BF16 && out_dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (batch < 1 || rows_per_batch < 0 || rows_per_batch > INT32_MAX || k < 32 || k % 32 != 0 || k > INT32_MAX)
    return GMM_ERR_SHAPE;
  if ((address(codes) | address(block_scale) | address(out)) % 16 != 0 || address(row_scale) % 4 != 0)
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (rows_per_batch == 0) return GMM_OK;
  const int64_t all_rows = int64_t(batch) * rows_per_batch;
  if (all_rows > INT32_MAX) return GMM_ERR_SHAPE;
  const DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(block_scale), row_scale,
                        rows_per_batch, k, out};
  const int64_t lanes = (k / (out_dtype == GMM_DTYPE_F32 ? 4 : 8) + 3) / 4;  // four pieces each
  const int threads = int(lanes >= kMaxThreads ? kMaxThreads : (lanes + 31) / 32 * 32);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned(all_rows);
  auto kern = out_dtype == GMM_DTYPE_F32
                  ? (nv ? dequantize_fp4_kernel<float, true> : dequantize_fp4_kernel<float, false>)
                  : (nv ? dequantize_fp4_kernel<__nv_bfloat16, true> : dequantize_fp4_kernel<__nv_bfloat16, false>);
  const cudaError_t e = launch_dependent(kern, grid, threads, 0, s, 1, p);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
