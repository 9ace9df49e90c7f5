// Grouped product of microscaled 4-bit rows with microscaled 4-bit weights on
// the block-scaled tensor cores:
//
//   out[r, c] = rs[r] ws[g, c] sum_b (a[r, b] w[g, c, b] sum_{kk in b} A(r, kk) W(g, c, kk)) + bias[g, c]
//
// tcgen05.mma.kind::mxf4nvf4 (NVFP4: an e4m3 scale per 16 k) or kind::mxf4
// (MXFP4: an E8M0 scale per 32 k), K = 64 codes an instruction, fp32
// accumulators in tensor memory.  Products of codes and scales are exact there;
// only the fp32 sums round.
//
// The weights are the M side (128 rows of n a tile) and up to 224 of a group's
// rows the N side, so a group of a few rows costs an MMA of N = 16 and the
// weights' bytes, and the output is written with n along the lanes.
//
// Scales reach tensor memory as the MMA wants them: for every 128 rows and 4
// bytes of scales (64 k of NVFP4, 128 k of MXFP4) lane l of the 32 lanes holds
// the 4 bytes of rows l, l + 32, l + 64 and l + 96.  A window of 16 scale bytes
// of 128 rows is stored as 2 KB in row order, so a bulk copy brings it from any
// first row, and a warp turns it into four such blocks in place: its lane l
// reads the 16 bytes of those four rows and writes the transposed 4 x 4 words.
// tcgen05.cp then copies each 512-byte block into tensor memory in order with
// the MMAs.
//
// Roles (288 threads): warp 0 TMA producer; warp 1 tensor memory and MMA; warps
// 2-5 epilogue; warps 6-8 turn the scales (128 weight rows, 2 x 128 rows).
// Tensor memory: two accumulators of 224 columns, 16 columns of weight scales
// and 32 of row scales.
#include <cuda_bf16.h>

#include <climits>
#include <cstdio>

#include "../../include/libgmm_moe.h"
#include "internal.h"
#include "ptx.cuh"
#include "worklist.cuh"

namespace gmmk {
namespace {

constexpr int BW = 128;       // weight rows a tile
constexpr int CHUNK = 224;    // most rows of a group a tile
constexpr int BK = 256;       // k a stage: 128 bytes of codes
constexpr int STAGES = 4;
constexpr int TBOX = 32;      // rows of one copy of row codes
constexpr int kThreads = 288;
constexpr int kMaxGroups = GMM_MAX_GROUPS;
constexpr uint32_t A_BYTES = BW * BK / 2;
constexpr uint32_t B_BYTES = CHUNK * BK / 2;
constexpr uint32_t TBOX_BYTES = TBOX * BK / 2;
constexpr uint32_t SF_BYTES = 128 * 16;  // a window of 128 rows' scales
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TM_SFA = 2 * CHUNK, TM_SFB = TM_SFA + 16;
static_assert(TM_SFB + 32 <= TMEM_COLS, "tensor memory budget");

constexpr uint32_t OFF_A = 0;
constexpr uint32_t OFF_B = OFF_A + STAGES * A_BYTES;
constexpr uint32_t OFF_SF = OFF_B + STAGES * B_BYTES;
constexpr uint32_t OFF_CTRL = OFF_SF + STAGES * 3 * SF_BYTES;
constexpr uint32_t OFF_FULL = OFF_CTRL;
constexpr uint32_t OFF_EMPTY = OFF_FULL + 8 * STAGES;
constexpr uint32_t OFF_TURNED = OFF_EMPTY + 8 * STAGES;
constexpr uint32_t OFF_ACCF = OFF_TURNED + 8 * STAGES;
constexpr uint32_t OFF_ACCE = OFF_ACCF + 16;
constexpr uint32_t OFF_DONE = OFF_ACCE + 16;
constexpr uint32_t OFF_TMEM = OFF_DONE + 8;
constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
constexpr uint32_t OFF_OFFS = OFF_CTRL + 256;
constexpr uint32_t OFF_TILES = OFF_OFFS + 4 * (kMaxGroups + 4);
constexpr uint32_t SMEM_BYTES = OFF_TILES + 4 * (kMaxGroups + 4) + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(OFF_ABORT + 4 <= OFF_OFFS, "control block overlaps the tables");

struct Params {
  const int32_t* group_sizes;
  int32_t num_total_groups, group_offset, num_local_groups;
  int32_t m, n, k;
  const uint8_t* lhs_scale;      // [windows, m, 16]
  const uint8_t* rhs_scale;      // [local groups, windows, n, 16]
  const float* lhs_row_scale;    // NULL or [m]
  const float* rhs_row_scale;    // NULL or [local groups, n]
  void* out;
  const void* bias;
  int32_t bias_f32;
  uint32_t* err;
};

__device__ __forceinline__ int32_t chunk_rows(const GemmTile& t) { return min(CHUNK, t.row_end - t.row0); }
__device__ __forceinline__ int32_t chunk_n(const GemmTile& t) { return (chunk_rows(t) + 15) & ~15; }

// Instruction descriptor of the block-scaled 4-bit kinds:
//   bits 4-5 B's scale id   bits 7-9 A format (1 = e2m1)   bits 10-11 B format (1 = e2m1)
//   bits 17-22 N >> 3   bit 23 scale format (0 = e4m3, 1 = E8M0)   bits 27-28 M >> 7
//   bits 29-30 A's scale id: the half word of the scales' column that a K = 64 step of MXFP4 reads
template <bool kNv>
__device__ __forceinline__ uint32_t idesc_fp4(int n, uint32_t scale_id) {
  return (scale_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | ((kNv ? 0u : 1u) << 23) | (1u << 27) |
         (scale_id << 29);
}

template <bool kNv>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 512 bytes of scales (32 lanes of 16 bytes) to 4 columns of tensor memory, in each of its four
// lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  // unswizzled: 8-lane groups of 128 bytes, 128 bytes apart
  const uint64_t desc = uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Turns the 128 rows of 16 scale bytes at `addr` into four 512-byte blocks, in place (one warp).
__device__ __forceinline__ void turn_scales(uint32_t addr, int lane) {
  const uint4 r0 = ld_shared_v4(addr + 16u * lane), r1 = ld_shared_v4(addr + 512u + 16u * lane),
              r2 = ld_shared_v4(addr + 1024u + 16u * lane), r3 = ld_shared_v4(addr + 1536u + 16u * lane);
  __syncwarp();
  st_shared_v4(addr + 16u * lane, r0.x, r1.x, r2.x, r3.x);
  st_shared_v4(addr + 512u + 16u * lane, r0.y, r1.y, r2.y, r3.y);
  st_shared_v4(addr + 1024u + 16u * lane, r0.z, r1.z, r2.z, r3.z);
  st_shared_v4(addr + 1536u + 16u * lane, r0.w, r1.w, r2.w, r3.w);
}

template <bool kNv, bool kOutF32>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tm_lhs, const __grid_constant__ CUtensorMap tm_rhs,
                    const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_ABORT);
  int32_t* offs = reinterpret_cast<int32_t*>(smem + OFF_OFFS);
  int32_t* tiles = reinterpret_cast<int32_t*>(smem + OFF_TILES);
  auto full_bar = [&](uint32_t s) { return sbase + OFF_FULL + 8 * s; };
  auto empty_bar = [&](uint32_t s) { return sbase + OFF_EMPTY + 8 * s; };
  auto turned_bar = [&](uint32_t s) { return sbase + OFF_TURNED + 8 * s; };
  auto accf_bar = [&](uint32_t b) { return sbase + OFF_ACCF + 8 * b; };
  auto acce_bar = [&](uint32_t b) { return sbase + OFF_ACCE + 8 * b; };
  const uint32_t done_bar = sbase + OFF_DONE;
  const int32_t go = p.group_offset;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(turned_bar(s), 3);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), 128);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch(&tm_lhs);
    tma_prefetch(&tm_rhs);
  }
  if (warp == 1) {
    tmem_alloc(sbase + OFF_TMEM, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 2) {
    build_group_offsets(p.group_sizes, p.num_total_groups, p.m, offs, p.err);
    build_tile_prefix(offs, go, p.num_local_groups, CHUNK, tiles);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM);

  const int32_t t_tiles = tiles[p.num_local_groups];
  const int32_t n_tiles = (p.n + BW - 1) / BW;
  const int32_t k_blocks = (p.k + BK - 1) / BK;
  const int32_t windows = (p.k + (kNv ? 255 : 511)) / (kNv ? 256 : 512);
  const int32_t total = t_tiles * n_tiles;
  // group by group, blocks of 16 chunks meeting the n tiles in turn: each weight tile comes from
  // memory once for the block, whose rows stay in L2
  auto item_of = [&](int32_t w) {
    return decode_gemm_tile(w, t_tiles, n_tiles, -16, tiles, offs, go, p.num_local_groups, CHUNK);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, pend_mask = 0;
      uint32_t pend_par[STAGES];
      bool ok = true;
      for (int32_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const GemmTile t = item_of(w);
        const int32_t nbox = (chunk_rows(t) + TBOX - 1) / TBOX;
        const int32_t n0 = t.n_tile * BW;
        const uint32_t sfa_bytes = uint32_t(min(BW, p.n - n0)) * 16u, sfb_bytes = uint32_t(chunk_rows(t)) * 16u;
        for (int32_t kb = 0; kb < k_blocks; ++kb) {
          if (!wait_bar(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_bar(stage);
          mbar_arrive_expect_tx(fb, A_BYTES + uint32_t(nbox) * TBOX_BYTES + sfa_bytes + sfb_bytes);
          const uint32_t b_dst = sbase + OFF_B + stage * B_BYTES, sf_dst = sbase + OFF_SF + stage * 3 * SF_BYTES;
          const int64_t win = kNv ? kb : kb >> 1;
          tma_load_3d(sbase + OFF_A + stage * A_BYTES, &tm_rhs, fb, kb * (BK / 2), n0, t.local_group);
          for (int32_t j = 0; j < nbox; ++j)
            tma_load_2d(b_dst + j * TBOX_BYTES, &tm_lhs, fb, kb * (BK / 2), t.row0 + TBOX * j);
          bulk_load(sf_dst, p.rhs_scale + ((t.local_group * int64_t(windows) + win) * p.n + n0) * 16, sfa_bytes, fb);
          bulk_load(sf_dst + SF_BYTES, p.lhs_scale + (win * p.m + t.row0) * 16, sfb_bytes, fb);
          pend_par[stage] = phase;
          pend_mask |= 1u << stage;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        for (int s = 0; s < STAGES; ++s)
          if (pend_mask >> s & 1u) drain_bar(full_bar(s), pend_par[s]);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
    bool ok = true;
    for (int32_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
      const GemmTile t = item_of(w);
      const int32_t ncols = chunk_n(t);
      if (!wait_bar(acce_bar(acc), acc_phase ^ 1u, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * CHUNK;
      for (int32_t kb = 0; kb < k_blocks; ++kb) {
        if (!wait_bar(full_bar(stage), phase, abort_flag, p.err) ||
            !wait_bar(turned_bar(stage), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t a0 = sbase + OFF_A + stage * A_BYTES;
          const uint32_t b0 = sbase + OFF_B + stage * B_BYTES;
          const uint32_t sf = sbase + OFF_SF + stage * 3 * SF_BYTES;
          // a stage uses 4 blocks of a window (NVFP4) or half of them (MXFP4)
          const int first = kNv ? 0 : 2 * (kb & 1);
#pragma unroll
          for (int j = 0; j < (kNv ? 4 : 2); ++j) {
            const uint32_t blk = 512u * uint32_t(first + j);
            copy_scales(tmem_base + TM_SFA + 4 * j, sf + blk);
            copy_scales(tmem_base + TM_SFB + 8 * j, sf + SF_BYTES + blk);
            if (ncols > 128) copy_scales(tmem_base + TM_SFB + 8 * j + 4, sf + 2 * SF_BYTES + blk);
          }
#pragma unroll
          for (int kk = 0; kk < BK / 64; ++kk) {
            const uint64_t ad = sw128_desc(a0 + kk * 32, 16, 1024);
            const uint64_t bd = sw128_desc(b0 + kk * 32, 16, 1024);
            const int j = kNv ? kk : kk >> 1;
            mma_fp4<kNv>(d_tmem, ad, bd, idesc_fp4<kNv>(ncols, kNv ? 0u : 2u * (kk & 1)), tmem_base + TM_SFA + 4 * j,
                         tmem_base + TM_SFB + 8 * j, (kb | kk) != 0 ? 1u : 0u);
          }
          mma_commit(empty_bar(stage));
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (lane == 0) mma_commit(accf_bar(acc));
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) {
      mma_commit(done_bar);
      drain_bar(done_bar, 0);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------------------------------------------------------- scales into the MMA's order
    const int part = warp - 6;  // the weights' 128 rows, the first and the second 128 of the chunk
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int32_t w = blockIdx.x; w < total && ok; w += gridDim.x) {
      const bool used = part < 2 || chunk_n(item_of(w)) > 128;
      for (int32_t kb = 0; kb < k_blocks; ++kb) {
        if (!wait_bar(full_bar(stage), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (used) {
          turn_scales(sbase + OFF_SF + stage * 3 * SF_BYTES + part * SF_BYTES, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(turned_bar(stage));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // TMEM lane = weight row = output column; TMEM column = row of the chunk.
    const int quarter = warp & 3;
    uint32_t acc = 0, acc_phase = 0;
    for (int32_t w = blockIdx.x; w < total; w += gridDim.x) {
      const GemmTile t = item_of(w);
      const int32_t rows = chunk_rows(t), ncols = chunk_n(t);
      const int32_t col = t.n_tile * BW + quarter * 32 + lane;
      const bool col_ok = col < p.n;
      float bias = 0.f, ws = 1.f;
      if (col_ok) {
        const int64_t bi = int64_t(t.local_group) * p.n + col;
        if (p.bias != nullptr)
          bias = p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + bi)
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[bi]);
        if (p.rhs_row_scale != nullptr) ws = __ldg(p.rhs_row_scale + bi);
      }
      if (!wait_bar(accf_bar(acc), acc_phase, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (uint32_t(quarter * 32) << 16) + acc * CHUNK;
#pragma unroll 1
      for (int32_t c0 = 0; c0 < ncols; c0 += 32) {
        uint32_t v[32];
        const float rs =
            p.lhs_row_scale != nullptr && c0 + lane < rows ? __ldg(p.lhs_row_scale + t.row0 + c0 + lane) : 1.f;
        tmem_ld_32cols(tbase + c0, v);
        if (c0 + 32 >= ncols) {
          tc_fence_before();
          mbar_arrive(acce_bar(acc));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float r = fmaf(__uint_as_float(v[i]) * __shfl_sync(0xffffffffu, rs, i), ws, bias);
          if (col_ok && c0 + i < rows) {
            const int64_t o = int64_t(t.row0 + c0 + i) * p.n + col;
            if constexpr (kOutF32)
              static_cast<float*>(p.out)[o] = r;
            else
              static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(r);
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    // Rows outside [offs[first local], offs[last local + 1]) are zero.
    const int64_t row_bytes = int64_t(p.n) * (kOutF32 ? 4 : 2);
    const int64_t lo_bytes = int64_t(offs[go]) * row_bytes;
    const int64_t hi_begin = int64_t(offs[go + p.num_local_groups]) * row_bytes;
    const int64_t n_lo = lo_bytes / 16;
    const int64_t n_all = n_lo + (int64_t(p.m) * row_bytes - hi_begin) / 16;
    const int64_t stride = int64_t(gridDim.x) * 128;
    for (int64_t i = int64_t(blockIdx.x) * 128 + (threadIdx.x - 64); i < n_all; i += stride) {
      const int64_t byte = i < n_lo ? i * 16 : hi_begin + (i - n_lo) * 16;
      st_global_v4(static_cast<uint8_t*>(p.out) + byte, 0u, 0u, 0u, 0u);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <bool kNv, bool kOutF32>
cudaError_t launch(const CUtensorMap& tm_lhs, const CUtensorMap& tm_rhs, const Params& p, int grid,
                   cudaStream_t stream) {
  auto kern = gemm_fp4_kernel<kNv, kOutF32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_BYTES));
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, SMEM_BYTES, stream>>>(tm_lhs, tm_rhs, p);
  return cudaGetLastError();
}

bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

}  // namespace
}  // namespace gmmk

extern "C" int gmm_fp4(const void* lhs_codes, const void* lhs_block_scale, const float* lhs_row_scale, int64_t m,
                       int64_t k, const void* rhs_codes, const void* rhs_block_scale, const float* rhs_row_scale,
                       int format, int32_t num_local_groups, int64_t n, const int32_t* group_sizes,
                       int32_t num_total_groups, int32_t group_offset, const void* rhs_bias, int bias_dtype, void* out,
                       int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace gmmk;
  if (rhs_codes == nullptr || rhs_block_scale == nullptr || group_sizes == nullptr ||
      (m > 0 && (lhs_codes == nullptr || lhs_block_scale == nullptr || out == nullptr)))
    return GMM_ERR_NULL;
  if (format != GMM_FP4_NVFP4 && format != GMM_FP4_MXFP4) return GMM_ERR_DTYPE;
  const bool nv = format == GMM_FP4_NVFP4;
  if (out_dtype != GMM_DTYPE_BF16 && out_dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (rhs_bias != nullptr && bias_dtype != GMM_DTYPE_BF16 && bias_dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (m < 0 || m > INT32_MAX || k < 32 || k > INT32_MAX || k % 32 != 0 || n < 8 || n > INT32_MAX || n % 8 != 0)
    return GMM_ERR_SHAPE;
  if (num_total_groups < 1 || num_total_groups > GMM_MAX_GROUPS || num_local_groups < 1 ||
      num_local_groups > num_total_groups)
    return GMM_ERR_SHAPE;
  if (group_offset < 0 || group_offset > num_total_groups - num_local_groups) return GMM_ERR_GROUP_OFFSET;
  if (((m + CHUNK - 1) / CHUNK + num_local_groups) * ((n + BW - 1) / BW) > INT32_MAX) return GMM_ERR_SHAPE;
  if (!aligned(lhs_codes, 16) || !aligned(lhs_block_scale, 16) || !aligned(rhs_codes, 16) ||
      !aligned(rhs_block_scale, 16) || !aligned(out, 16) || !aligned(lhs_row_scale, 4) || !aligned(rhs_row_scale, 4) ||
      !aligned(rhs_bias, bias_dtype == GMM_DTYPE_F32 ? 4 : 2) || !aligned(group_sizes, 4))
    return GMM_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < GMM_WORKSPACE_MIN_BYTES || !aligned(workspace, 16))
    return GMM_ERR_WORKSPACE;
  int sms = 0;
  if (int st = require_device(&sms)) return st;
  if (m == 0) return GMM_OK;
  CUtensorMap tm_lhs, tm_rhs;
  {
    const uint64_t dims[2] = {uint64_t(k / 2), uint64_t(m)};
    const uint32_t box[2] = {BK / 2, TBOX};
    if (int st = byte_map(&tm_lhs, 2, lhs_codes, dims, box)) return st;
  }
  {
    const uint64_t dims[3] = {uint64_t(k / 2), uint64_t(n), uint64_t(num_local_groups)};
    const uint32_t box[3] = {BK / 2, BW, 1};
    if (int st = byte_map(&tm_rhs, 3, rhs_codes, dims, box)) return st;
  }
  const Params p{group_sizes, num_total_groups, group_offset, num_local_groups, int32_t(m), int32_t(n), int32_t(k),
                 static_cast<const uint8_t*>(lhs_block_scale), static_cast<const uint8_t*>(rhs_block_scale),
                 lhs_row_scale, rhs_row_scale, out, rhs_bias, bias_dtype == GMM_DTYPE_F32 ? 1 : 0,
                 static_cast<uint32_t*>(workspace)};
  if (call_log_enabled())
    std::fprintf(stderr, "libgmm: gmm_fp4 m=%lld k=%lld n=%lld groups=%d local=%d offset=%d format=%s out=%s\n",
                 (long long)m, (long long)k, (long long)n, num_total_groups, num_local_groups, group_offset,
                 nv ? "nvfp4" : "mxfp4", out_dtype == GMM_DTYPE_F32 ? "f32" : "bf16");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = out_dtype == GMM_DTYPE_F32;
  const cudaError_t e = nv ? (f32 ? launch<true, true>(tm_lhs, tm_rhs, p, sms, s)
                                  : launch<true, false>(tm_lhs, tm_rhs, p, sms, s))
                           : (f32 ? launch<false, true>(tm_lhs, tm_rhs, p, sms, s)
                                  : launch<false, false>(tm_lhs, tm_rhs, p, sms, s));
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
