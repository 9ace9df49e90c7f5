// Tokens' rows sorted by expert, and back with the router's weights, with
// their gradients.
//
//   sort      a stable counting sort of the tokens * topk slots by expert
//   dispatch  out[rows[t, j]] = x[t]
//   combine   out[t] = sum_j w[t, j] in[rows[t, j]]
//   its gradients  din[rows[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], in[rows[t, j]]>
//
// All but the sort are bound by memory: they go token by token, so that what
// is shared by a token's slots (x[t], dout[t]) is read once, and the expert
// order is only ever the address of whole rows.
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "../../include/libgmm_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

// The row of a slot as a call is given it; anything that is no row of the order counts as dropped.
__device__ __forceinline__ int32_t slot_row(const int32_t* rows, int64_t slot, int64_t slots) {
  const int32_t r = __ldg(rows + slot);
  return r < slots ? r : -1;
}

// ------------------------------------------------------------------ the sort
// One cluster of CTAs.  Every warp owns a run of consecutive slots: it counts its
// experts in its own row of a table in shared memory, the table is summed down
// the warps and across the CTAs (each CTA writes its sums into all of them, so
// that one barrier of the cluster is all they wait for), and then the warp walks
// its run again and gives each slot the next place of its expert, equal experts
// within a step of 32 in lane order.  So the order is stable and no result hangs
// on the order of an atomic.  Dropped slots count as one more expert after the
// last.
//
// Bound by latency, not by its 12 bytes a slot: 32768 slots of 128 experts take
// 6.6 us in a graph, 12000 cycles, of which 4000 are the three barriers of the
// cluster and the sums between them and 4000 the last walk, whose stores are
// scattered.  There lanes with equal experts find each other by a ballot for each
// bit of the expert's number (with __match_any_sync, and the sums read from the
// other CTAs instead of written into them, 7.6 us).
constexpr int kSortCluster = 16;

// kWarps a CTA; `run` slots a warp, a multiple of 32; 2^bits > num_experts.
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
    sort_kernel(const int32_t* __restrict__ experts, int32_t slots, int32_t num_experts, int32_t bits, int32_t run,
                int32_t* __restrict__ group_sizes, int32_t* __restrict__ rows, int32_t* __restrict__ source,
                int32_t ctas) {
  constexpr int kThreads = 32 * kWarps;
  griddep_begin();
  experts = after_begin(experts);
  extern __shared__ uint32_t table[];  // [kWarps][bins]; each CTA's sums [ctas][bins]; first places [bins]
  __shared__ uint32_t warp_sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bins = num_experts + 1;
  uint32_t* mine = table + warp * bins;
  uint32_t* sums = table + kWarps * bins;
  uint32_t* place = sums + ctas * bins;
  const int32_t rank = ctas > 1 ? int32_t(cluster_ctarank()) : 0;
  const int64_t first = int64_t(rank * kWarps + warp) * run;
  const int32_t lo = int32_t(first < slots ? first : slots);
  const int32_t hi = int32_t(first + run < slots ? first + run : slots);
  // the run's first four steps stay in registers
  int32_t held[4];
  auto bin_of = [&](int32_t e) { return e >= 0 && e < num_experts ? e : num_experts; };
#pragma unroll
  for (int i = 0; i < 4; ++i) held[i] = lo + 32 * i + lane < hi ? bin_of(__ldg(experts + lo + 32 * i + lane)) : -1;
  for (int b = lane; b < bins; b += 32) mine[b] = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (held[i] >= 0) atomicAdd(mine + held[i], 1u);
  for (int32_t s = lo + 128 + lane; s < hi; s += 32) atomicAdd(mine + bin_of(__ldg(experts + s)), 1u);
  __syncthreads();
  if (ctas > 1) cluster_sync();  // every CTA has started: its shared memory can be written
  for (int b = tid; b < bins; b += kThreads) {
    uint32_t c[kWarps], sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c[w] = table[w * bins + b];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      table[w * bins + b] = sum;
      sum += c[w];
    }
    if (ctas > 1) {
      const uint32_t to = smem_u32(sums + rank * bins + b);
      for (int r = 0; r < ctas; ++r) st_shared_cluster_u32(mapa_shared(to, uint32_t(r)), sum);
    } else {
      sums[b] = sum;
    }
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  // Each expert's rows over all CTAs, those of the CTAs before this one, and the experts before: a
  // thread takes kPer consecutive experts.
  constexpr int kPer = GMM_MAX_GROUPS / kThreads;
  uint32_t all[kPer], before[kPer], sum = 0;
  const int b0 = tid * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    all[i] = before[i] = 0;
    if (b0 + i < num_experts) {
      for (int r = 0; r < ctas; ++r) {
        const uint32_t c = sums[r * bins + b0 + i];
        all[i] += c;
        before[i] += r < rank ? c : 0u;
      }
      if (rank == 0) group_sizes[b0 + i] = int32_t(all[i]);
    }
    sum += all[i];
  }
  uint32_t incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t start = incl - sum, kept = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    start += w < warp ? warp_sums[w] : 0u;
    kept += warp_sums[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (b0 + i < num_experts) place[b0 + i] = start + before[i];
    start += all[i];
  }
  if (tid == kThreads - 1) {  // the dropped ones
    for (int r = 0; r < rank; ++r) kept += sums[r * bins + num_experts];
    place[num_experts] = kept;
  }
  __syncthreads();
  auto put = [&](int32_t s, int32_t b) {  // a step of 32 slots, b the bin of slot s or -1
    uint32_t same = __ballot_sync(0xffffffffu, b >= 0);
    for (int i = 0; i < bits; ++i) {
      const bool set = (b >> i) & 1;
      const uint32_t with = __ballot_sync(0xffffffffu, set);
      same &= set ? with : ~with;
    }
    const int ahead = __popc(same & ((1u << lane) - 1u));
    const uint32_t at = b >= 0 ? place[b] + mine[b] + uint32_t(ahead) : 0u;
    __syncwarp();
    if (b >= 0) {
      if (ahead == 0) mine[b] += uint32_t(__popc(same));
      rows[s] = b < num_experts ? int32_t(at) : -1;
      source[at] = b < num_experts ? s : -1;
    }
    __syncwarp();
  };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lo + 32 * i < hi) put(lo + 32 * i + lane, held[i]);
  for (int32_t s0 = lo + 128; s0 < hi; s0 += 32)
    put(s0 + lane, s0 + lane < hi ? bin_of(__ldg(experts + s0 + lane)) : -1);
}

template <int kWarps>
cudaError_t launch_sort_as(const int32_t* experts, int32_t slots, int32_t num_experts, int32_t* group_sizes,
                           int32_t* rows, int32_t* source, int ctas, cudaStream_t stream) {
  const size_t smem = size_t(kWarps + ctas + 1) * (num_experts + 1) * sizeof(uint32_t);
  int bits = 1;
  while ((1 << bits) <= num_experts) ++bits;
  auto kern = sort_kernel<kWarps>;
  cudaError_t e = cudaSuccess;
  // A launch may use 48 KB unasked, its static shared memory (under 1 KB here) among them.  The setting is
  // the kernel's, not the launch's: always the most that any call needs, so that no call takes from another
  // thread's what that one has just been allowed.
  constexpr size_t kMost = size_t(kWarps + kSortCluster + 1) * (GMM_MAX_GROUPS + 1) * sizeof(uint32_t);
  static_assert(kMost <= 226 * 1024, "shared memory budget");
  if (smem > 47 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost));
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t warps = int64_t(ctas) * kWarps;
  const int32_t run = int32_t(((slots + warps - 1) / warps + 31) / 32 * 32);
  return launch_dependent(kern, unsigned(ctas), 32 * kWarps, smem, stream, ctas, experts, slots, num_experts, bits,
                          run, group_sizes, rows, source, int32_t(ctas));
}

// Up to 1024 slots: one CTA of 8 warps (256 slots 2.4 us in a graph, 1024 slots 3.2; with 32 warps
// 4.1); up to 2048 one CTA of 32 (4.7 us, with eight CTAs 5.2); up to 8192 eight CTAs (the portable
// cluster; 4096 slots 5.4 us, with one 6.1), above that sixteen (32768 slots 6.6 us, with eight 7.3).
cudaError_t launch_sort(const int32_t* experts, int32_t slots, int32_t num_experts, int32_t* group_sizes,
                        int32_t* rows, int32_t* source, cudaStream_t stream) {
  if (slots <= 1024)
    return launch_sort_as<8>(experts, slots, num_experts, group_sizes, rows, source, 1, stream);
  const int ctas = slots <= 2048 ? 1 : slots <= 8192 ? 8 : kSortCluster;
  return launch_sort_as<32>(experts, slots, num_experts, group_sizes, rows, source, ctas, stream);
}

// ------------------------------------------------------------------ rows of any width
// A row is moved in units of 16, 8, 4 or 2 bytes, the widest that every row's
// address and width are a multiple of; a unit holds kN elements.
template <class U, class T>
struct Unit {
  static constexpr int kN = int(sizeof(U) / sizeof(T));
  static __device__ __forceinline__ void unpack(U u, float (&f)[kN]) {
    T t[kN];
    memcpy(t, &u, sizeof(U));
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = float(t[i]);
  }
  static __device__ __forceinline__ U pack(const float (&f)[kN]) {
    U u;
    if constexpr (std::is_same<T, float>::value) {
      memcpy(&u, f, sizeof(U));
    } else if constexpr (kN == 1) {
      const T t = __float2bfloat16_rn(f[0]);
      memcpy(&u, &t, sizeof(U));
    } else {
      __nv_bfloat162 t[kN / 2];
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) t[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&u, t, sizeof(U));
    }
    return u;
  }
};

constexpr int kThreads = 128;

// Units a lane moves at a time: `bytes` of them whatever their width.
template <class U>
constexpr int units_of(int bytes) {
  return int(sizeof(U)) > bytes ? 1 : bytes / int(sizeof(U));
}

template <class U>
__device__ __forceinline__ U zero_unit() {
  U u;
  memset(&u, 0, sizeof(U));
  return u;
}

// One warp for each token and run of 32 * kPer units of its row.
template <class U, int kPer>
__global__ void __launch_bounds__(kThreads)
    dispatch_kernel(const U* __restrict__ x, int64_t tokens, int64_t units, int64_t x_units, int32_t topk,
                    int64_t parts, const int32_t* __restrict__ rows, const int32_t* __restrict__ source,
                    U* __restrict__ out) {
  griddep_begin();
  x = after_begin(x), rows = after_begin(rows), source = after_begin(source);
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / parts;
  if (t >= tokens) return;
  const int64_t c0 = (w - t * parts) * (32 * kPer) + lane;
  const int32_t r = lane < topk ? slot_row(rows, t * topk + lane, tokens * topk) : -1;
  const int32_t s = lane < topk ? __ldg(source + t * topk + lane) : 0;
  U v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (c0 + 32 * i < units) v[i] = __ldg(x + t * x_units + c0 + 32 * i);
  for (int j = 0; j < topk; ++j) {
    const int32_t to = __shfl_sync(0xffffffffu, r, j);
    if (to >= 0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c0 + 32 * i < units) out[to * units + c0 + 32 * i] = v[i];
    }
    if (__shfl_sync(0xffffffffu, s, j) < 0) {  // row t * topk + j is past the groups
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c0 + 32 * i < units) out[(t * topk + j) * units + c0 + 32 * i] = zero_unit<U>();
    }
  }
}

template <class U, class T, int kPer, int kBatch, int kCta>
__global__ void __launch_bounds__(kCta)
    combine_kernel(const U* __restrict__ in, int64_t tokens, int64_t units, int32_t topk, int64_t parts,
                   const int32_t* __restrict__ rows, const float* __restrict__ weights, U* __restrict__ out) {
  griddep_begin();
  in = after_begin(in), rows = after_begin(rows), weights = after_begin(weights);
  constexpr int N = Unit<U, T>::kN;
  const int lane = threadIdx.x & 31;
  const int64_t w = int64_t(blockIdx.x) * (kCta / 32) + (threadIdx.x >> 5);
  const int64_t t = w / parts;
  if (t >= tokens) return;
  const int64_t c0 = (w - t * parts) * (32 * kPer) + lane;
  const int32_t r = lane < topk ? slot_row(rows, t * topk + lane, tokens * topk) : -1;
  const float g = lane < topk && weights != nullptr ? __ldg(weights + t * topk + lane) : 1.f;
  float acc[kPer][N];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[i][n] = 0.f;
  // kBatch rows are on their way before the first is used
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    U got[kBatch][kPer];
    float gj[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int32_t from = __shfl_sync(0xffffffffu, r, (j0 + q) & 31);  // -1 past the last slot
      gj[q] = __shfl_sync(0xffffffffu, g, (j0 + q) & 31);
      const bool there = j0 + q < topk && from >= 0;
      gj[q] = there ? gj[q] : 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        got[q][i] = there && c0 + 32 * i < units ? __ldg(in + from * units + c0 + 32 * i) : zero_unit<U>();
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float f[N];
        Unit<U, T>::unpack(got[q][i], f);
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] = fmaf(gj[q], f[n], acc[i][n]);
      }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (c0 + 32 * i < units) out[t * units + c0 + 32 * i] = Unit<U, T>::pack(acc[i]);
}

// The sums over the warp of one or two values: of two, the first in the lower half of the lanes and the
// second in the upper, as the halves exchange what they do not go on with.
template <int kBatch>
__device__ __forceinline__ float warp_sums(const float (&sum)[kBatch], int lane) {
  static_assert(kBatch == 1 || kBatch == 2);
  const bool high = kBatch == 2 && (lane & 16);
  float v = (high ? sum[kBatch - 1] : sum[0]) + __shfl_xor_sync(0xffffffffu, high ? sum[0] : sum[kBatch - 1], 16);
#pragma unroll
  for (int k = 8; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}

// One CTA for each token: its warps share the row's columns, 32 * kPer consecutive
// ones at a time; their parts of the dot products are summed in warp order.
// kBatch of the token's rows are on their way at once.  Bound by memory and, of
// narrow units, by the instructions a unit takes: columns that are all there are
// not asked for one by one (8192 tokens, 2 rows of 4096 bf16: 53 us for 50; 4096
// tokens, 8 rows of 2048: 45 for 42; 2000 tokens, 6 rows of 7168: 60 for 55; 3001
// tokens, 5 rows of 1027 f32: 27 for 20; a first form, 512 threads with strided
// columns, took 59, 50, 85 and 32).
template <class U, class T, int kPer, int kBatch, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
    combine_backward_kernel(const U* __restrict__ dout, const U* __restrict__ in, int64_t tokens, uint32_t units,
                            int32_t topk,
                            const int32_t* __restrict__ rows, const int32_t* __restrict__ source,
                            const float* __restrict__ weights, U* __restrict__ din, float* __restrict__ dweights) {
  griddep_begin();
  dout = after_begin(dout), in = after_begin(in), rows = after_begin(rows), source = after_begin(source);
  weights = after_begin(weights);
  constexpr int N = Unit<U, T>::kN;
  __shared__ float part[kWarps][GMM_MAX_TOPK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int32_t r = lane < topk ? slot_row(rows, t * topk + lane, tokens * topk) : -1;
  const int32_t s = lane < topk ? __ldg(source + t * topk + lane) : 0;
  const float g = lane < topk ? __ldg(weights + t * topk + lane) : 0.f;
  const uint32_t gone = __ballot_sync(0xffffffffu, s < 0);  // rows of these numbers are past the groups
  part[warp][lane] = 0.f;
  __syncwarp();
  // A warp's 32 * kPer columns from c0 - lane on, all of them the row's (kFull) or not.
  auto columns = [&](uint32_t c0, auto full) {
    constexpr bool kFull = decltype(full)::value;
    float d[kPer][N];
    const U* pd = dout + t * units + c0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      Unit<U, T>::unpack(kFull || c0 + 32 * i < units ? __ldg(pd + 32 * i) : zero_unit<U>(), d[i]);
    for (int j0 = 0; j0 < topk; j0 += kBatch) {
      U got[kBatch][kPer];
      int32_t row[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int32_t from = __shfl_sync(0xffffffffu, r, (j0 + q) & 31);
        row[q] = j0 + q < topk ? from : -1;
        const U* p = in + int64_t(row[q]) * units + c0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          got[q][i] = row[q] >= 0 && (kFull || c0 + 32 * i < units) ? __ldg(p + 32 * i) : zero_unit<U>();
      }
      float sum[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const float gj = __shfl_sync(0xffffffffu, g, (j0 + q) & 31);
        sum[q] = 0.f;
        U* p = din + int64_t(row[q]) * units + c0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          float f[N], o[N];
          Unit<U, T>::unpack(got[q][i], f);
#pragma unroll
          for (int n = 0; n < N; ++n) sum[q] = fmaf(d[i][n], f[n], sum[q]), o[n] = gj * d[i][n];
          if (row[q] >= 0 && (kFull || c0 + 32 * i < units)) p[32 * i] = Unit<U, T>::pack(o);
        }
      }
      const float all = warp_sums<kBatch>(sum, lane);
      const int j = j0 + lane / (32 / kBatch);
      if (lane % (32 / kBatch) == 0 && j < topk) part[warp][j] += all;
    }
    for (uint32_t left = gone; left != 0; left &= left - 1) {
      U* p = din + (t * topk + __ffs(left) - 1) * units + c0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (kFull || c0 + 32 * i < units) p[32 * i] = zero_unit<U>();
    }
  };
  for (uint32_t c0 = warp * (32 * kPer); c0 < units; c0 += blockDim.x * kPer) {
    if (c0 + 32 * kPer <= units)
      columns(c0 + lane, std::true_type{});
    else
      columns(c0 + lane, std::false_type{});
  }
  __syncthreads();
  if (int(threadIdx.x) < topk) {
    float sum = 0.f;
    for (uint32_t w = 0; w < blockDim.x / 32; ++w) sum += part[w][threadIdx.x];
    dweights[t * topk + threadIdx.x] = r >= 0 ? sum : 0.f;  // r is this slot's row; a dropped one's sum may be 0 * inf
  }
}

// go(unit) for the widest unit type that `bits` (addresses and pitches in bytes, or-ed) allows.
template <class F>
cudaError_t by_unit(uint64_t bits, F&& go) {
  if (bits % 16 == 0) return go(uint4{});
  if (bits % 8 == 0) return go(uint2{});
  if (bits % 4 == 0) return go(uint32_t{});
  return go(uint16_t{});
}

uint64_t address(const void* p) { return uint64_t(reinterpret_cast<uintptr_t>(p)); }

int check(int dtype, int64_t tokens, int64_t d, int32_t topk) {
  if (dtype != GMM_DTYPE_BF16 && dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (tokens < 0 || d < 1 || d > INT32_MAX || topk < 1 || topk > GMM_MAX_TOPK || tokens > kMaxSize / topk)
    return GMM_ERR_SHAPE;
  return GMM_OK;
}

// Warps of `per` units a lane over every token's row, as a grid of CTAs of so many threads; 0: too large.
unsigned row_grid(int64_t tokens, int64_t units, int per, int threads, int64_t* parts) {
  *parts = (units + 32 * per - 1) / (32 * per);
  const int64_t blocks = (tokens * *parts + threads / 32 - 1) / (threads / 32);
  return blocks <= INT32_MAX ? unsigned(blocks) : 0u;
}

int done(cudaError_t e) { return e == cudaSuccess ? GMM_OK : record_cuda_error(e); }

template <class T>
cudaError_t combine(const void* in, int64_t tokens, int64_t d, int32_t topk, const int32_t* rows,
                    const float* weights, void* out, cudaStream_t s) {
  return by_unit(address(in) | address(out) | uint64_t(d) * sizeof(T), [&](auto unit) -> cudaError_t {
    using U = decltype(unit);
    if constexpr (sizeof(U) < sizeof(T)) {
      return cudaErrorInvalidValue;  // excluded by the alignment check
    } else {
      const int64_t units = d * int64_t(sizeof(T)) / int64_t(sizeof(U));
      int64_t parts;
      // Wide units: 32 bytes a lane, four rows at once of more than two; where the sums are many, 64 bytes, two
      // rows and CTAs of two warps (8192 tokens, 2 rows of 4096 bf16 31.5 us, with 128 threads 33.5, as few
      // tokens 34; 4096 tokens, 8 rows of 2048 25.3, as few 26.4; but 8192 tokens, 8 rows of 1032, with some
      // lanes of a token's last run idle, 33.0, as few 32.0; 64 tokens, 4 rows of 2048 2.0 us in a graph, as
      // many tokens 2.2; 8 MB lie between that and the others).  Narrow units: 24 bytes, 128 threads (8192 tokens, 8 rows of 1027 bf16 37 us,
      // with 32 bytes 49 and with 8 39; 3001 tokens, 5 rows of 1027 f32 12.5 us, with 32 bytes 13.1 and with
      // 16 14.6; 8192 tokens, 2 rows of 2047 f32 32 us, with 64 threads 48).
      auto go = [&](auto per, auto batch, auto threads) -> cudaError_t {
        const unsigned grid = row_grid(tokens, units, per, threads, &parts);
        if (grid == 0) return cudaErrorInvalidConfiguration;
        return launch_dependent(combine_kernel<U, T, per, batch, threads>, grid, threads, 0, s, 1,
                                static_cast<const U*>(in), tokens, units, topk, parts, rows, weights,
                                static_cast<U*>(out));
      };
      constexpr std::integral_constant<int, units_of<U>(sizeof(U) == 16 ? 32 : 24)> per;
      constexpr std::integral_constant<int, kThreads> threads;
      constexpr std::integral_constant<int, 2> two;
      constexpr std::integral_constant<int, 4> four;
      if constexpr (sizeof(U) == 16) {
        if (tokens * units >= (8 << 20) / 16)
          return go(std::integral_constant<int, units_of<U>(64)>{}, two, std::integral_constant<int, 64>{});
      }
      return topk <= 2 ? go(per, two, threads) : go(per, four, threads);
    }
  });
}

template <class T>
cudaError_t combine_backward(const void* dout, const void* in, int64_t tokens, int64_t d, int32_t topk,
                             const int32_t* rows, const int32_t* source, const float* weights, void* din,
                             float* dweights, cudaStream_t s) {
  return by_unit(address(dout) | address(in) | address(din) | uint64_t(d) * sizeof(T), [&](auto unit) -> cudaError_t {
    using U = decltype(unit);
    if constexpr (sizeof(U) < sizeof(T)) {
      return cudaErrorInvalidValue;
    } else {
      const int64_t units = d * int64_t(sizeof(T)) / int64_t(sizeof(U));
      // 32 bytes a thread, two rows at once where there are two (8192 tokens, 2 rows of 4096 bf16 53 us, one
      // at once 54.5; 2000 tokens, 6 rows of 7168 60 and 67; 8192 tokens, one row of 2048 21 and 19).  Narrow
      // units: one row, 24 bytes, 16 of 2-byte units (8192 tokens, 8 rows of 1030 bf16 50 us, with 16 bytes
      // 66, with 32 68, two rows of 16 63; 8 rows of 1027 72, with 32 bytes 81, two rows of 16 83).
      constexpr bool kWide = sizeof(U) == 16;
      constexpr int kPer = units_of<U>(kWide ? 32 : sizeof(U) == 2 ? 16 : 24);
      // 4 warps a token leave the fewest idle at a token's ends; tokens that do not fill the SMs with them
      // (8 CTAs on each of 152) have as many as the row has columns for, up to 16 (8 rows of 7168 bf16:
      // 64 tokens 6 us, with four warps 14; 608 tokens 24, with four 29; 1216 tokens 49 with either)
      const bool few = tokens <= 8 * 152;
      const int64_t warps = (units + 32 * kPer - 1) / (32 * kPer), most = few ? 16 : 4;
      auto kern = few ? combine_backward_kernel<U, T, kPer, 1, 16> : combine_backward_kernel<U, T, kPer, 1, 4>;
      if constexpr (kWide) {
        if (topk > 1) kern = few ? combine_backward_kernel<U, T, kPer, 2, 16> : combine_backward_kernel<U, T, kPer, 2, 4>;
      }
      return launch_dependent(kern, unsigned(tokens), 32 * unsigned(warps < most ? warps : most), 0, s, 1,
                              static_cast<const U*>(dout), static_cast<const U*>(in), tokens, uint32_t(units), topk,
                              rows, source, weights, static_cast<U*>(din), dweights);
    }
  });
}

}  // namespace
}  // namespace gmmk

extern "C" int gmm_sort_by_expert(const int32_t* experts, int64_t tokens, int32_t topk, int32_t num_experts,
                                  int32_t* group_sizes, int32_t* rows, int32_t* source, void* stream) {
  using namespace gmmk;
  if (num_experts < 1 || num_experts > GMM_MAX_GROUPS) return GMM_ERR_SHAPE;
  if (int st = check(GMM_DTYPE_F32, tokens, 1, topk)) return st;
  if (group_sizes == nullptr || (tokens > 0 && (experts == nullptr || rows == nullptr || source == nullptr)))
    return GMM_ERR_NULL;
  if ((address(experts) | address(group_sizes) | address(rows) | address(source)) % 4 != 0) return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  return done(launch_sort(experts, int32_t(tokens * topk), num_experts, group_sizes, rows, source,
                          static_cast<cudaStream_t>(stream)));
}

extern "C" int gmm_dispatch(const void* x, int dtype, int64_t tokens, int64_t d, int64_t x_ld, int32_t topk,
                            const int32_t* rows, const int32_t* source, void* out, void* stream) {
  using namespace gmmk;
  if (int st = check(dtype, tokens, d, topk)) return st;
  if (x_ld < d) return GMM_ERR_SHAPE;
  if (tokens > 0 && (x == nullptr || rows == nullptr || source == nullptr || out == nullptr))
    return GMM_ERR_NULL;
  const uint64_t el = dtype == GMM_DTYPE_F32 ? 4 : 2;
  if ((address(x) | address(out)) % el != 0 || (address(rows) | address(source)) % 4 != 0) return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(by_unit(address(x) | address(out) | uint64_t(d) * el | uint64_t(x_ld) * el, [&](auto unit) -> cudaError_t {
    using U = decltype(unit);
    const int64_t units = d * int64_t(el) / int64_t(sizeof(U));
    int64_t parts;
    constexpr int kPer = units_of<U>(32);
    const unsigned grid = row_grid(tokens, units, kPer, kThreads, &parts);
    if (grid == 0) return cudaErrorInvalidConfiguration;
    return launch_dependent(dispatch_kernel<U, kPer>, grid, kThreads, 0, s, 1, static_cast<const U*>(x), tokens, units,
                            x_ld * int64_t(el) / int64_t(sizeof(U)), topk, parts, rows, source, static_cast<U*>(out));
  }));
}

extern "C" int gmm_combine(const void* in, int dtype, int64_t tokens, int64_t d, int32_t topk, const int32_t* rows,
                           const float* weights, void* out, void* stream) {
  using namespace gmmk;
  if (int st = check(dtype, tokens, d, topk)) return st;
  if (tokens > 0 && (in == nullptr || rows == nullptr || out == nullptr))
    return GMM_ERR_NULL;
  if ((address(in) | address(out)) % (dtype == GMM_DTYPE_F32 ? 4 : 2) != 0 ||
      (address(rows) | address(weights)) % 4 != 0)
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(dtype == GMM_DTYPE_F32 ? combine<float>(in, tokens, d, topk, rows, weights, out, s)
                                     : combine<__nv_bfloat16>(in, tokens, d, topk, rows, weights, out, s));
}

extern "C" int gmm_combine_backward(const void* dout, const void* in, int dtype, int64_t tokens, int64_t d,
                                    int32_t topk, const int32_t* rows, const int32_t* source, const float* weights,
                                    void* din, float* dweights, void* stream) {
  using namespace gmmk;
  if (int st = check(dtype, tokens, d, topk)) return st;
  if (tokens > 0 && (dout == nullptr || in == nullptr || rows == nullptr || source == nullptr || weights == nullptr || din == nullptr || dweights == nullptr))
    return GMM_ERR_NULL;
  if ((address(dout) | address(in) | address(din)) % (dtype == GMM_DTYPE_F32 ? 4 : 2) != 0 ||
      (address(rows) | address(source) | address(weights) | address(dweights)) % 4 != 0)
    return GMM_ERR_ALIGN;
  if (int st = require_device(nullptr)) return st;
  if (tokens == 0) return GMM_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(dtype == GMM_DTYPE_F32
                  ? combine_backward<float>(dout, in, tokens, d, topk, rows, source, weights, din, dweights, s)
                  : combine_backward<__nv_bfloat16>(dout, in, tokens, d, topk, rows, source, weights, din, dweights,
                                                    s));
}
