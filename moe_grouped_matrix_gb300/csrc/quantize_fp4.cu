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
// quotient of two short significands.  The fp32 quotients used here round, but
// never onto or across a point half way between two codes (or two e4m3 values)
// unless the exact quotient is that point: were a numerator one unit of 2^-23
// off the half-way product, the quotient would be more than half a unit off the
// half-way point, because the point's significand is over half of the
// numerator's.  So codes and scales are those of exact arithmetic.
//
// Bound by memory: 2 bytes read and 9/16 written per value (17/32 for MXFP4).
#include <cuda_bf16.h>

#include <climits>

#include "../../include/libgmm_moe.h"
#include "internal.h"

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

// The least e with a <= limit * 2^(e + shift), limit in [0.5, 1) * 2^0, for finite a > 0.
__device__ __forceinline__ int least_exponent(float a, float limit, int shift) {
  int x;
  const float f = frexpf(a, &x);
  return x - shift + (f > limit ? 1 : 0);
}

// 16 consecutive values as fp32.
__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
    v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <class T>
__device__ __forceinline__ void load_values(const T* p, bool wide, float (&v)[16]) {
  if (wide) {
    load16(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = load1(p + i);
  }
}

// Largest magnitude as bits; above 0x7F800000 - 1 when one is not finite.
__device__ __forceinline__ uint32_t amax16(const float (&v)[16]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return a;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// Codes of 16 values divided by s > 0, in 8 bytes.
__device__ __forceinline__ uint2 encode16(const float (&v)[16], float s) {
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[8 * h + i], s);
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out[h])
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  }
  return make_uint2(out[0], out[1]);
}

// Codes of zeros: the signs alone.
__device__ __forceinline__ uint2 signs16(const float (&v)[16]) {
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) out[i / 8] |= (__float_as_uint(v[i]) >> 31) << (4 * (i % 8) + 3);
  return make_uint2(out[0], out[1]);
}

// kThreadsPerRow threads quantise one input row and write it to its rows of the
// result.  A thread takes 16 values at a time: a block of NVFP4, half a block
// of MXFP4 (its neighbour lane has the other half).
template <class T, bool kNv, int kThreadsPerRow>
__global__ void __launch_bounds__(kMaxThreads) quantize_fp4_kernel(const QuantParams p, bool wide) {
  __shared__ uint32_t warp_max[kMaxThreads / 32];
  __shared__ int32_t to_rows[kMaxThreads / kThreadsPerRow][GMM_MAX_TOPK], zero_rows[kMaxThreads / kThreadsPerRow][GMM_MAX_TOPK];
  constexpr int kRows = kMaxThreads / kThreadsPerRow;
  const int tid = threadIdx.x % kThreadsPerRow, sub = threadIdx.x / kThreadsPerRow;
  const int64_t row = int64_t(blockIdx.x) * kRows + sub;
  const bool there = row < p.in_rows;
  const int64_t out_rows = p.rows_per_batch * p.topk;  // of one batch's matrix
  const int64_t batch = there ? row / p.rows_per_batch : 0;
  if (there && tid < p.topk) {
    int32_t r = 0, z = -1;
    if (p.rows != nullptr) {
      const int64_t slot = row * p.topk + tid;
      r = __ldg(p.rows + slot);
      r = r < out_rows ? r : -1;
      z = __ldg(p.source + slot) < 0 ? int32_t(slot) : -1;
    } else {
      r = int32_t(row - batch * p.rows_per_batch);
    }
    to_rows[sub][tid] = r;
    zero_rows[sub][tid] = z;
  }
  __syncthreads();
  const T* x = static_cast<const T*>(p.x) + (there ? row * p.ld : 0);
  const int64_t units = there ? p.k / 16 : 0;
  float row_scale = 1.f, up = 1.f;
  if constexpr (kNv) {
    uint32_t high = 0;
    for (int64_t u = tid; u < units; u += kThreadsPerRow) {
      float v[16];
      load_values(x + 16 * u, wide, v);
      const uint32_t a = amax16(v);
      if (a < kInfBits) high = max(high, a);
    }
    high = __reduce_max_sync(0xffffffffu, high);
    if constexpr (kThreadsPerRow > 32) {
      if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = high;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreadsPerRow / 32; ++w) high = max(high, warp_max[sub * (kThreadsPerRow / 32) + w]);
    }
    if (high != 0) {
      // 6 * 448 = 0.65625 * 2^12
      const int e = max(least_exponent(__uint_as_float(high), 0.65625f, 12), -126);
      row_scale = exp2_int(e), up = exp2_int(-e);
    }
  }
  const int64_t windows = (units + (kNv ? 15 : 31)) / (kNv ? 16 : 32);
  const int64_t padded = windows * (kNv ? 16 : 32);  // threads past the row's end write the windows' zeros
  const int64_t batch_rows = p.in_rows / p.rows_per_batch > 1 ? p.rows_per_batch : out_rows;
  uint8_t* scale = p.scale + batch * windows * batch_rows * 16;
  uint8_t* codes = p.codes + batch * batch_rows * (p.k / 2);
  const int64_t steps = there ? (padded + kThreadsPerRow - 1) / kThreadsPerRow : 0;
  for (int64_t step = 0; step < steps; ++step) {
    const int64_t u = step * kThreadsPerRow + tid;
    float v[16];
    uint32_t a = 0;
    if (u < units) {
      load_values(x + 16 * u, wide, v);
      a = amax16(v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    uint32_t byte;
    float s;
    if constexpr (kNv) {
      if (a >= kInfBits) {
        byte = 0x7Fu, s = 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= up;
        const float q = __fdiv_rn(__uint_as_float(a) * up, 6.f);
        uint16_t e8;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.f), "f"(q));
        byte = e8 & 0xFFu;
        // e4m3 back to fp32: 3 bits after the point, exponent bias 7, subnormals below 2^-6
        s = byte >= 8 ? __uint_as_float((byte << 20) + (120u << 23)) : float(byte) * 0x1p-9f;
      }
    } else {
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      if (a >= kInfBits) {
        byte = 255u, s = 0.f;
      } else if (a == 0) {
        byte = 0u, s = 0.f;
      } else {
        // 6 = 0.75 * 2^3
        const int e = max(least_exponent(__uint_as_float(a), 0.75f, 3), -127);
        byte = uint32_t(e + 127);
        s = e < -126 ? 0x1p-127f : exp2_int(e);
      }
    }
    uint2 c = make_uint2(0u, 0u);
    if (a < kInfBits) c = s > 0.f ? encode16(v, s) : signs16(v);
    for (int j = 0; j < p.topk; ++j) {
      const int32_t r = to_rows[sub][j], z = zero_rows[sub][j];
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        const int32_t to = pass == 0 ? r : z;
        if (to < 0) continue;
        if (u < units)
          *reinterpret_cast<uint2*>(codes + to * (p.k / 2) + 8 * u) = pass == 0 ? c : make_uint2(0u, 0u);
        const int64_t b = kNv ? u : u / 2;  // the block
        if (u < padded && (kNv || (u & 1) == 0))
          scale[((b / 16) * batch_rows + to) * 16 + b % 16] = pass == 0 ? uint8_t(u < units ? byte : 0u) : uint8_t(0);
      }
    }
  }
  if constexpr (kNv) {
    if (there && tid < p.topk) {
      const int32_t r = to_rows[sub][tid], z = zero_rows[sub][tid];
      if (r >= 0) p.row_scale[batch * batch_rows + r] = row_scale;
      if (z >= 0) p.row_scale[z] = 1.f;
    }
  }
}

struct DequantParams {
  const uint8_t* codes;
  const uint8_t* scale;
  const float* row_scale;
  int64_t rows_per_batch, k, units;  // units: 16 values each, over all rows
  void* out;
};

// The value of a scale byte.
template <bool kNv>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if constexpr (kNv) {
    const uint32_t m = b & 0x7Fu;
    if (m == 0x7Fu) return __uint_as_float(0x7FC00000u);
    const float s = m >= 8 ? __uint_as_float((m << 20) + (120u << 23)) : float(m) * 0x1p-9f;
    return b & 0x80u ? -s : s;
  } else {
    if (b == 255u) return __uint_as_float(0x7FC00000u);
    return b == 0 ? 0x1p-127f : __uint_as_float(b << 23);
  }
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  // 0, 0.5, 1, 1.5, 2, 3, 4, 6: an exponent of 2 bits with bias 1 and one bit after the point
  const uint32_t m = c & 7u;
  const float v = m >= 2 ? __uint_as_float((m << 22) + (126u << 23)) : 0.5f * float(m);
  return c & 8u ? -v : v;
}

template <class T, bool kNv>
__global__ void __launch_bounds__(kMaxThreads) dequantize_fp4_kernel(const DequantParams p) {
  const int64_t i = int64_t(blockIdx.x) * kMaxThreads + threadIdx.x;
  if (i >= p.units) return;
  const int64_t per_row = p.k / 16, row = i / per_row, u = i - row * per_row;
  const int64_t batch = row / p.rows_per_batch, r = row - batch * p.rows_per_batch;
  const int64_t b = kNv ? u : u / 2, windows = (p.k + (kNv ? 255 : 511)) / (kNv ? 256 : 512);
  const float s = scale_value<kNv>(p.scale[((batch * windows + b / 16) * p.rows_per_batch + r) * 16 + b % 16]);
  const float rs = kNv ? __ldg(p.row_scale + row) : 1.f;
  const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.codes + row * (p.k / 2)) + u);
  const uint32_t w[2] = {c.x, c.y};
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = e2m1_value(w[j / 8] >> (4 * (j % 8))) * s * rs;
  if constexpr (sizeof(T) == 4) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + 16 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      memcpy(&h[j], &q, 4);
    }
    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + 16 * i);
    o[0] = make_uint4(h[0], h[1], h[2], h[3]);
    o[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

template <class T, bool kNv>
cudaError_t quantize(const QuantParams& p, cudaStream_t s) {
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ld * sizeof(T) % 16 == 0;
  // Rows of up to 1024 values: one warp each, 8 rows a block; longer rows: a block each.
  const bool narrow = p.k <= 1024;
  const int64_t blocks = narrow ? (p.in_rows + 7) / 8 : p.in_rows;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (narrow)
    quantize_fp4_kernel<T, kNv, 32><<<unsigned(blocks), kMaxThreads, 0, s>>>(p, wide);
  else
    quantize_fp4_kernel<T, kNv, kMaxThreads><<<unsigned(blocks), kMaxThreads, 0, s>>>(p, wide);
  return cudaGetLastError();
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
  const int64_t units = int64_t(batch) * rows_per_batch * (k / 16);
  const int64_t blocks = (units + kMaxThreads - 1) / kMaxThreads;
  if (blocks > INT32_MAX) return GMM_ERR_SHAPE;
  const DequantParams p{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(block_scale), row_scale,
                        rows_per_batch, k, units, out};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = unsigned(blocks);
  if (out_dtype == GMM_DTYPE_F32) {
    if (nv) dequantize_fp4_kernel<float, true><<<grid, kMaxThreads, 0, s>>>(p);
    else dequantize_fp4_kernel<float, false><<<grid, kMaxThreads, 0, s>>>(p);
  } else {
    if (nv) dequantize_fp4_kernel<__nv_bfloat16, true><<<grid, kMaxThreads, 0, s>>>(p);
    else dequantize_fp4_kernel<__nv_bfloat16, false><<<grid, kMaxThreads, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
