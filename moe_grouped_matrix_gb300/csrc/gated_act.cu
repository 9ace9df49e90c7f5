// The gated activation between an expert's two products, and its gradient:
//   out = act(g) u,   dg = d u act'(g),   du = d act(g),   [g | u] = a row of h.
//
// Elementwise, bound by memory: 6 bytes an output in bf16 forward, 10 backward (32768 rows
// of 1024: 28.9 us and 48.1, 6.9 TB/s; 3001 rows of 2051 f32 13.6 and 20.2, 5.4 and 6.1).
// A thread handles whole units of a row, the largest (up to 16 bytes) that all rows of all
// operands are aligned to; a block is some rows, so that no index is divided (few wide rows keep few
// SMs busy: 8 rows of 14336 bf16 3.3 us and 4.4, 256 rows 9.4 and 10.4).  bf16 results
// take an exponential and a quotient of few instructions: with expf() and a full division
// the instructions were the bound, not memory (39.5 us forward).
#include <cuda_bf16.h>

#include <climits>

#include "activation.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kThreads = 256;

// The values of a unit U of elements T.
template <class U, class T>
struct Values {
  static constexpr int kN = int(sizeof(U) / sizeof(T));
  float v[kN];
  __device__ __forceinline__ explicit Values(const U& raw) {
    const T* t = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = float(t[i]);
  }
  __device__ __forceinline__ Values() {}
  __device__ __forceinline__ U pack() const {
    U raw;
    T* t = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int i = 0; i < kN; ++i) t[i] = T(v[i]);
    return raw;
  }
};

// A unit of two bytes or more as the integer that moves it.
template <int kBytes>
struct UnitOf;
template <>
struct UnitOf<16> { using type = uint4; };
template <>
struct UnitOf<8> { using type = uint2; };
template <>
struct UnitOf<4> { using type = uint32_t; };
template <>
struct UnitOf<2> { using type = uint16_t; };

struct Params {
  const char* dout;  // backward only
  const char* h;
  char* out;
  int64_t rows, ld;  // row pitch of h in bytes
  int64_t f;         // bytes of half a row
  int32_t units;     // of half a row
};

// Blocks of x units by 256 / x rows or fewer; a thread takes kPer units of its row at a time.
template <class U, class T, int kAct, int kPer, bool kBack>
__global__ void __launch_bounds__(kThreads) gated_kernel(Params p) {
  griddep_begin();
  p.h = after_begin(p.h), p.dout = after_begin(p.dout);
  constexpr bool kFast = sizeof(T) == 2;
  const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;
  const U* g = reinterpret_cast<const U*>(p.h + row * p.ld);
  const U* u = reinterpret_cast<const U*>(p.h + row * p.ld + p.f);
  const U* d = reinterpret_cast<const U*>(p.dout + row * p.f);
  U* out = reinterpret_cast<U*>(p.out + row * p.f * (kBack ? 2 : 1));
  U* out_u = reinterpret_cast<U*>(p.out + row * p.f * 2 + p.f);
  const int step = blockDim.x;
  for (int c0 = threadIdx.x; c0 < p.units; c0 += step * kPer) {
    U gs[kPer], us[kPer], ds[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = c0 + i * step;
      if (c < p.units) {
        gs[i] = __ldg(g + c), us[i] = __ldg(u + c);
        if constexpr (kBack) ds[i] = __ldg(d + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = c0 + i * step;
      if (c >= p.units) break;
      Values<U, T> gv(gs[i]), uv(us[i]);
      if constexpr (kBack) {
        Values<U, T> dv(ds[i]);
#pragma unroll
        for (int j = 0; j < Values<U, T>::kN; ++j) {
          float slope;
          const float a = act_value<kAct, kFast>(gv.v[j], slope);
          gv.v[j] = dv.v[j] * uv.v[j] * slope;
          uv.v[j] = dv.v[j] * a;
        }
        out[c] = gv.pack(), out_u[c] = uv.pack();
      } else {
#pragma unroll
        for (int j = 0; j < Values<U, T>::kN; ++j) gv.v[j] = act_value<kAct, kFast>(gv.v[j]) * uv.v[j];
        out[c] = gv.pack();
      }
    }
  }
}

template <int kBytes, class T, bool kBack>
cudaError_t launch(Params p, int act, cudaStream_t stream) {
  using U = typename UnitOf<kBytes>::type;
  // two units of 16 bytes or four of fewer on their way (four and two: gradient 49.3 us for 48.1 in bf16, f32 rows
  // of 2051 16.0 for 13.6)
  constexpr int kPer = kBytes == 16 ? 2 : 4;
  p.units = int32_t(p.f / kBytes);
  // whole warps of a row that its units divide among evenly, over as many turns as 256 threads need
  const int turns = (p.units + kThreads * kPer - 1) / (kThreads * kPer);
  int x = ((p.units + turns * kPer - 1) / (turns * kPer) + 31) / 32 * 32;
  if (p.units <= 16 * kPer) {  // short rows: parts of a warp
    x = 1;
    while (x * kPer < p.units) x *= 2;
  }
  const int y = kThreads / x;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(unsigned(x), unsigned(y));
  cfg.gridDim = dim3(unsigned((p.rows + y - 1) / y));
  cfg.stream = stream;
  cudaLaunchAttribute at[1]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  return act == GMM_ACT_SILU ? cudaLaunchKernelEx(&cfg, gated_kernel<U, T, GMM_ACT_SILU, kPer, kBack>, p)
                             : cudaLaunchKernelEx(&cfg, gated_kernel<U, T, GMM_ACT_GELU, kPer, kBack>, p);
}

template <bool kBack>
int gated(const void* dout, const void* h, int dtype, int64_t rows, int64_t f, int64_t h_ld, int act, void* out,
          void* stream) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (rows < 0 || rows > kMaxSize || f < 1 || f > kMaxSize / 8 || h_ld < 2 * f ||
      (act != GMM_ACT_SILU && act != GMM_ACT_GELU))
    return GMM_ERR_SHAPE;
  if (rows > 0 && (h == nullptr || out == nullptr || (kBack && dout == nullptr))) return GMM_ERR_NULL;
  const int size = dtype == GMM_DTYPE_F32 ? 4 : 2;
  // what all rows of all operands are aligned to
  const uintptr_t all = reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(out) |
                        reinterpret_cast<uintptr_t>(dout) | uintptr_t(f * size) | (rows > 1 ? uintptr_t(h_ld * size) : 0);
  if (all % size != 0) return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (rows == 0) return GMM_OK;
  const Params p{static_cast<const char*>(dout), static_cast<const char*>(h), static_cast<char*>(out), rows,
                 h_ld * size, f * size, 0};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == GMM_DTYPE_F32) {
    e = all % 16 == 0 ? launch<16, float, kBack>(p, act, s)
        : all % 8 == 0 ? launch<8, float, kBack>(p, act, s) : launch<4, float, kBack>(p, act, s);
  } else {
    e = all % 16 == 0 ? launch<16, __nv_bfloat16, kBack>(p, act, s)
        : all % 8 == 0 ? launch<8, __nv_bfloat16, kBack>(p, act, s)
        : all % 4 == 0 ? launch<4, __nv_bfloat16, kBack>(p, act, s) : launch<2, __nv_bfloat16, kBack>(p, act, s);
  }
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}

}  // namespace
}  // namespace gmmk

extern "C" int gmm_gated_act(const void* h, int dtype, int64_t rows, int64_t f, int64_t h_ld, int act, void* out,
                             void* stream) {
  return gmmk::gated<false>(nullptr, h, dtype, rows, f, h_ld, act, out, stream);
}

extern "C" int gmm_gated_act_backward(const void* dout, const void* h, int dtype, int64_t rows, int64_t f, int64_t h_ld,
                                      int act, void* dh, void* stream) {
  return gmmk::gated<true>(dout, h, dtype, rows, f, h_ld, act, dh, stream);
}
