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
// The weights are the MMA's M side and a group's rows its N side, so a group of
// a few rows costs an MMA of N = 16 or 32 and the weights' bytes.  One kernel,
// two shapes:
//   pair   256 weight rows on an SM pair (tcgen05.mma.cta_group::2), 128 in each
//          CTA, by up to 224 rows of a group, half of them in each CTA's shared
//          memory.  Two accumulators of 224 columns, 16 columns of weight scales
//          and 32 of row scales take 496 of the 512 columns of tensor memory;
//          256 rows would leave one accumulator, and every tile would wait for
//          the epilogue of the one before.
//   single 128 weight rows on one SM by up to 32 rows: for groups of a few rows,
//          where the time is the reading of the weights and what counts is how much
//          of them is on its way (64 rows and a stage less: 66.2 us against 64.2).
//
// Scales reach tensor memory as the MMA wants them: for every 128 rows and 4
// bytes of scales (64 k of NVFP4, 128 k of MXFP4) lane l of 32 holds the 4 bytes
// of rows l, l + 32, l + 64 and l + 96.  A window of 16 scale bytes of 128 rows
// is stored as 2 KB in row order, so a bulk copy brings it from any first row,
// and a warp turns it into four such blocks in place: its lane l reads the 16
// bytes of those four rows and writes the transposed 4 x 4 words.  tcgen05.cp
// then copies each 512-byte block into tensor memory in order with the MMAs; in
// a pair the leader's copy moves both CTAs' blocks, each into its own memory.
// In a pair each CTA holds the scales of its own weight rows and of all the
// chunk's rows.
//
// Each role is a warp of its own, and every loop is uniform over its warp (waits
// end in a vote, tiles are broadcast), so that addresses and descriptors stay in
// uniform registers: with one lane's own loop each tensor-core instruction and
// each copy took some 80 cycles to issue, a stage over 1300 for 420 cycles of
// MMA.  For the same reason a warp turns the whole of a stage, and has stages of
// its own.  Codes and scales have rings of their own: a window of scales is ready
// later than the codes copied with it, and is cheap to hold (prefill with one
// ring of 5 for both 658 us, with 7 windows 617, with 8 or 9 the same, with 4 767).
//
// Measured (L2 cold): 8 experts, 16384 rows, 4096 -> 28672: NVFP4 605 us, 6.4
// PFLOP/s; MXFP4 562 us.  128 experts, 32768 rows, 2048 -> 2048: 83 us for 456 MB
// (67 us at the copy rate).  Decoding, 64 experts, 256 rows, 4096 -> 2048: 52 us
// for 303 MB (45 us), 46 back to back with the rows' quantisation.  What bounds
// the first is the way from L2 to the SMs: its tiles bring 8.5 GB of codes and 1.5
// of scales into shared memory, 34.9 KB a CTA and stage, which at the 62 bytes a
// cycle that an SM takes by TMA are 563 of a stage's about 600 cycles, beside 420
// of MMA (10.0 GB at 18 TB/s: 557 us; 4 experts, 8192 rows, 4096 -> 8192: 1.43 GB
// counted, as planned, in 94 us).  For seconds on end it is the power cap (700 us).
//
// Roles (512 threads): warp 0 copies codes; warp 1 tensor memory and MMA (the
// leader's in a pair); warps 2-9 epilogue, each set of four every other 32 rows;
// warp 10 copies scales; warps 11-15 turn them.
#include <cuda_bf16.h>

#include <climits>
#include <cstdio>
#include <utility>

#include "../../include/libgmm_moe.h"
#include "internal.h"
#include "ptx.cuh"
#include "worklist.cuh"

namespace gmmk {
namespace {

constexpr int BW = 128;   // weight rows a CTA
constexpr int BK = 256;   // k a stage: 128 bytes of codes
constexpr int kThreads = 512;
constexpr int kTurners = 5;
constexpr int kMaxGroups = GMM_MAX_GROUPS;
constexpr uint32_t ROW_BYTES = BK / 2;
constexpr uint32_t A_BYTES = BW * ROW_BYTES;
constexpr uint32_t SF_BYTES = 128 * 16;  // a window of 128 rows' scales
constexpr uint32_t OUT_PITCH = 80;       // of 32 bf16 columns in an epilogue warp's buffer: no bank conflicts
constexpr uint32_t OUT_BYTES = 16 * OUT_PITCH;

template <bool kPair>
struct Shape {
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTileW = kCtas * BW;          // weight rows a tile
  static constexpr int kChunk = kPair ? 224 : 32;    // most rows of a group a tile
  static constexpr int kUnit = kPair ? 32 : 16;      // rows a chunk is a multiple of
  static constexpr int kRows = kChunk / kCtas;       // of them in a CTA's shared memory
  static constexpr int kParts = kPair ? 3 : 2;       // 128-row windows of scales: weights, rows
  static constexpr int kStages = kPair ? 5 : 8;   // of codes
  static constexpr int kScales = kPair ? 7 : 8;   // of scales
  static constexpr uint32_t B_BYTES = kRows * ROW_BYTES;
  static constexpr uint32_t TM_SFA = 2 * kChunk, TM_SFB = TM_SFA + 16;
  static constexpr uint32_t kColumns = kPair ? 512 : 256;  // TM_SFB + 4 * 8 (4 * 4) columns, to a power of two
  static constexpr uint32_t OFF_A = 0;
  static constexpr uint32_t OFF_B = OFF_A + kStages * A_BYTES;
  static constexpr uint32_t OFF_SF = OFF_B + kStages * B_BYTES;
  static constexpr uint32_t OFF_OUT = OFF_SF + kScales * kParts * SF_BYTES;
  static constexpr uint32_t OFF_CTRL = OFF_OUT + 8 * OUT_BYTES;
  static constexpr uint32_t OFF_FULL = OFF_CTRL;                   // codes (of both CTAs, the leader's)
  static constexpr uint32_t OFF_EMPTY = OFF_FULL + 8 * kStages;    // the MMA's commit
  static constexpr uint32_t OFF_SFULL = OFF_EMPTY + 8 * kStages;   // this CTA's scales
  static constexpr uint32_t OFF_TURNED = OFF_SFULL + 8 * kScales;  // scales turned (of both CTAs, the leader's)
  static constexpr uint32_t OFF_SEMPTY = OFF_TURNED + 8 * kScales; // the MMA's commit
  static constexpr uint32_t OFF_ACCF = OFF_SEMPTY + 8 * kScales;
  static constexpr uint32_t OFF_ACCE = OFF_ACCF + 16;
  static constexpr uint32_t OFF_DONE = OFF_ACCE + 16;
  static constexpr uint32_t OFF_TMEM = OFF_DONE + 8;
  static constexpr uint32_t OFF_ABORT = OFF_TMEM + 4;
  static constexpr uint32_t OFF_UNWIND = OFF_ABORT + 4;  // the follower's: the leader has given up
  static constexpr uint32_t OFF_ISSUED = OFF_UNWIND + 4; // stages whose codes this CTA's copies were issued for
  static constexpr uint32_t OFF_TURNS = OFF_ISSUED + 4;  // times each window of scales has been turned
  static constexpr uint32_t OFF_SIGNAL = (OFF_TURNS + 4 * kScales + 15) / 16 * 16;  // 16 bytes, see signal_leader
  static constexpr uint32_t OFF_OFFS = OFF_CTRL + 512;
  static constexpr uint32_t OFF_TILES = OFF_OFFS + 4 * (kMaxGroups + 4);
  static constexpr uint32_t SMEM_BYTES = OFF_TILES + 4 * (kMaxGroups + 4) + 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
  static_assert(OFF_SIGNAL + 16 <= OFF_OFFS, "control block overlaps the tables");
  static_assert(B_BYTES % 1024 == 0 && OFF_SF % 1024 == 0, "swizzle atoms");
  static_assert(TM_SFB + (kPair ? 32 : 16) <= kColumns, "tensor memory budget");
};

struct Params {
  const int32_t* group_sizes;
  int32_t num_total_groups, group_offset, num_local_groups;
  int32_t m, n, k;
  const uint8_t* lhs_scale;    // [windows, m, 16]
  const uint8_t* rhs_scale;    // [local groups, windows, n, 16]
  const float* lhs_row_scale;  // NULL or [m]
  const float* rhs_row_scale;  // NULL or [local groups, n]
  void* out;
  const void* bias;
  int32_t bias_f32;
  uint32_t* err;
};

// Maps of the row codes in boxes of 64, 32 and 16 rows: a CTA's rows of a chunk,
// a multiple of 16 up to 112, take three copies at most.
struct Maps {
  CUtensorMap rhs, lhs64, lhs32, lhs16;
};

__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A wait of a whole warp, with one answer for all of it.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* err) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, err));
}
__device__ __forceinline__ bool wait_warp_cluster(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                                  uint32_t* err) {
  return __all_sync(0xffffffffu, wait_bar_cluster(bar, parity, abort_flag, err));
}

__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Instruction descriptor of the block-scaled 4-bit kinds:
//   bits 4-5 B's scale id   bits 7-9 A format (1 = e2m1)   bits 10-11 B format (1 = e2m1)
//   bits 17-22 N >> 3   bit 23 scale format (0 = e4m3, 1 = E8M0)   bits 27-28 M >> 7
//   bits 29-30 A's scale id: the half word of the scales' column that a K = 64 step of MXFP4 reads
template <bool kNv>
__device__ __forceinline__ uint32_t idesc_fp4(int m, int n, uint32_t scale_id) {
  return (scale_id << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | ((kNv ? 0u : 1u) << 23) |
         (uint32_t(m >> 7) << 27) | (scale_id << 29);
}

#define GMM_MMA_FP4(group, kind)                                                                              \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::" group ".kind::" kind \
               " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                             \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                \
               : "memory")

template <bool kPair, bool kNv>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (kPair && kNv) GMM_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (kPair && !kNv) GMM_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
  if constexpr (!kPair && kNv) GMM_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
  if constexpr (!kPair && !kNv) GMM_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
}
#undef GMM_MMA_FP4

// 512 bytes of scales (32 lanes of 16 bytes: unswizzled, 8-lane groups of 128 bytes one after the
// other) to 4 columns of tensor memory, in each of its four lane quarters.
template <bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
  if constexpr (kPair)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool kPair>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (kPair)
    mma_commit_pair(bar, 0x3);
  else
    mma_commit(bar);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Tells the leader that this CTA's scales of a stage are turned: a copy of 16 bytes to the same place
// there, whose bytes count on the leader's barrier.  The order that is relied on: each lane's turned
// scales, its proxy fence, the warp's synchronisation, this copy (of the async proxy, so after the fence),
// the copy's completion (a release at cluster scope on the barrier), the leader's wait (an acquire), the
// tcgen05.cp that reads the scales.  Each step but one is documented as such: that the completion's
// release carries, beside the copy itself, what precedes the copy.  An mbarrier arrive with release at
// cluster scope would not need that step, but it takes 1570 cycles for this copy's 140: prefill 752 us
// for 596, 128 experts 104 for 84; with a warp for each window 698 and 102, with 8 windows 662 and 96.
constexpr uint32_t kSignalBytes = 16;
__device__ __forceinline__ void signal_leader(uint32_t addr, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          mapa_shared(addr, 0)),
      "r"(addr), "r"(kSignalBytes), "r"(mapa_shared(bar, 0))
      : "memory");
}

// Turns kParts windows of 128 rows of 16 scale bytes into four 512-byte blocks each, in place (one warp).
template <int kParts>
__device__ __forceinline__ void turn_scales(uint32_t addr, int lane) {
  uint4 r[kParts][4];
#pragma unroll
  for (int w = 0; w < kParts; ++w)
#pragma unroll
    for (int q = 0; q < 4; ++q) r[w][q] = ld_shared_v4(addr + w * SF_BYTES + 512u * q + 16u * lane);
  __syncwarp();
#pragma unroll
  for (int w = 0; w < kParts; ++w) {
    const uint32_t a = addr + w * SF_BYTES + 16u * lane;
    st_shared_v4(a, r[w][0].x, r[w][1].x, r[w][2].x, r[w][3].x);
    st_shared_v4(a + 512u, r[w][0].y, r[w][1].y, r[w][2].y, r[w][3].y);
    st_shared_v4(a + 1024u, r[w][0].z, r[w][1].z, r[w][2].z, r[w][3].z);
    st_shared_v4(a + 1536u, r[w][0].w, r[w][1].w, r[w][2].w, r[w][3].w);
  }
}

// 16 lanes by 32 columns of tensor memory: registers 4g, 4g + 1 hold lane t / 4 and columns
// 8g + 2 (t % 4) and the next, 4g + 2, 4g + 3 the same of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Four 8 x 8 matrices of 16-bit values, stored transposed: register j of thread t holds matrix j's
// column t / 4 of rows 2 (t % 4) and the next; lane 8j + r gives the address of its row r.
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ float load_bias(const Params& p, int64_t i) {
  return p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + i)
                    : __bfloat162float(static_cast<const __nv_bfloat16*>(p.bias)[i]);
}

template <bool kPair, bool kNv, bool kOutF32>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp4_kernel(const __grid_constant__ Maps maps, Params p) {
  using S = Shape<kPair>;
  constexpr int kStages = S::kStages, kScales = S::kScales;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = uniform(int32_t(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int32_t pair = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int32_t npairs = kPair ? gridDim.x >> 1 : gridDim.x;
  auto word = [&](uint32_t off) { return reinterpret_cast<volatile uint32_t*>(smem + off); };
  volatile uint32_t* abort_flag = word(S::OFF_ABORT);
  int32_t* offs = reinterpret_cast<int32_t*>(smem + S::OFF_OFFS);
  int32_t* tiles = reinterpret_cast<int32_t*>(smem + S::OFF_TILES);
  auto full_bar = [&](uint32_t s) { return sbase + S::OFF_FULL + 8 * s; };
  auto empty_bar = [&](uint32_t s) { return sbase + S::OFF_EMPTY + 8 * s; };
  auto sfull_bar = [&](uint32_t s) { return sbase + S::OFF_SFULL + 8 * s; };
  auto turned_bar = [&](uint32_t s) { return sbase + S::OFF_TURNED + 8 * s; };
  auto sempty_bar = [&](uint32_t s) { return sbase + S::OFF_SEMPTY + 8 * s; };
  auto accf_bar = [&](uint32_t b) { return sbase + S::OFF_ACCF + 8 * b; };
  auto acce_bar = [&](uint32_t b) { return sbase + S::OFF_ACCE + 8 * b; };
  const uint32_t done_bar = sbase + S::OFF_DONE;
  const int32_t go = p.group_offset;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);             // the (leader's) expect_tx; bytes of both CTAs of a pair
      mbar_init(empty_bar(s), 1);            // the MMA's commit, to both CTAs of a pair
    }
    for (int s = 0; s < kScales; ++s) {
      mbar_init(sfull_bar(s), 1);            // this CTA's expect_tx
      mbar_init(turned_bar(s), 1);           // the leader's turning warp; in a pair the follower's signal
      mbar_init(sempty_bar(s), 1);           // the MMA's commit, to both CTAs of a pair
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);             // the MMA's commit, to both CTAs of a pair
      mbar_init(acce_bar(b), 8 * S::kCtas);  // one lane of each epilogue warp
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0u;
    *word(S::OFF_UNWIND) = 0u;
    for (int s = 0; s < kScales; ++s) word(S::OFF_TURNS)[s] = 0u;
    fence_mbar_init();
    tma_prefetch(&maps.rhs);
    tma_prefetch(&maps.lhs16);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(sbase + S::OFF_TMEM, S::kColumns);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(sbase + S::OFF_TMEM, S::kColumns);
      tmem_relinquish();
    }
  }
  griddep_begin();
  p.group_sizes = after_begin(p.group_sizes), p.bias = after_begin(p.bias);
  p.lhs_row_scale = after_begin(p.lhs_row_scale), p.rhs_row_scale = after_begin(p.rhs_row_scale);
  if (warp == 2) {
    build_group_offsets(p.group_sizes, p.num_total_groups, p.m, offs, p.err);
    build_tile_prefix(offs, go, p.num_local_groups, S::kChunk, tiles);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = uniform(*word(S::OFF_TMEM));

  const int32_t t_tiles = uniform(tiles[p.num_local_groups]);
  const int32_t n_tiles = (p.n + S::kTileW - 1) / S::kTileW;
  const int32_t k_blocks = (p.k + BK - 1) / BK;
  const int32_t windows = (p.k + (kNv ? 255 : 511)) / (kNv ? 256 : 512);
  const int32_t total = t_tiles * n_tiles;
  // This CTA's (pair's) items: w = pair, pair + npairs, ...
  const int32_t items = pair < total ? (total - 1 - pair) / npairs + 1 : 0;
  // Group by group, blocks of 16 chunks meeting the n tiles in turn: each weight tile comes from
  // memory once for the block, whose rows stay in L2.  A group's units of rows are spread evenly
  // over its chunks, so that no tile is left with a few.
  auto lane_tile = [&](int32_t item) {
    constexpr int32_t kBlock = 16;
    const int32_t w = pair + item * npairs;
    GemmTile t;
    t.local_group = find_group(tiles, p.num_local_groups, w / n_tiles);
    const int32_t g0 = tiles[t.local_group], chunks = tiles[t.local_group + 1] - g0;
    const int32_t r = w - g0 * n_tiles;                            // item within the group
    const int32_t b0 = r / (kBlock * n_tiles) * kBlock;            // first chunk of its block
    const int32_t width = min(kBlock, chunks - b0), rb = r - b0 * n_tiles;
    t.n_tile = rb / width;
    const int32_t i = b0 + rb - t.n_tile * width;                  // chunk of the group
    const int32_t start = offs[go + t.local_group], end = offs[go + t.local_group + 1];
    const int32_t units = (end - start + S::kUnit - 1) / S::kUnit, base = units / chunks, more = units - base * chunks;
    t.row0 = start + (i * base + min(i, more)) * S::kUnit;
    t.row_end = min(end, t.row0 + (base + (i < more ? 1 : 0)) * S::kUnit);
    return t;
  };
  // The tile of an item, for a whole warp that asks for one item after the other: every 32 items
  // each lane works out one of them, which takes the divisions and the search out of each tile's
  // way (some 100 cycles for every stage of 16).
  GemmTile mine{};
  auto tile_of = [&](int32_t item) {
    const int at = item & 31;
    if (at == 0 && item + lane < items) mine = lane_tile(item + lane);
    return GemmTile{__shfl_sync(0xffffffffu, mine.local_group, at), __shfl_sync(0xffffffffu, mine.row0, at),
                    __shfl_sync(0xffffffffu, mine.row_end, at), __shfl_sync(0xffffffffu, mine.n_tile, at)};
  };
  auto chunk_n = [](const GemmTile& t) { return (t.row_end - t.row0 + S::kUnit - 1) / S::kUnit * S::kUnit; };
  // bytes of one CTA's copies of codes in a stage of tile t
  auto code_bytes = [&](const GemmTile& t) { return A_BYTES + uint32_t(chunk_n(t) / S::kCtas) * ROW_BYTES; };

  uint32_t issued = 0;  // warps that copy: stages of the sequence whose copies were issued (and armed)
  if (warp == 0) {
    // ---------------------------------------------------------------- copies of codes (both CTAs)
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    const uint32_t full0 = kPair ? mapa_shared(full_bar(0), 0) : full_bar(0);
    for (int32_t item = 0; item < items && ok; ++item) {
      const GemmTile t = tile_of(item);
      const int32_t rows = chunk_n(t) / S::kCtas;  // of the chunk that this CTA holds
      const int32_t trow = t.row0 + int32_t(rank) * rows;
      const int32_t wrow = t.n_tile * S::kTileW + int32_t(rank) * BW;
      const uint32_t bytes = S::kCtas * code_bytes(t);
      for (int32_t kb = 0; kb < k_blocks; ++kb) {
        if (!wait_warp(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (elected()) {
          if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes);
          const uint32_t fb = full0 + 8 * stage;
          const int32_t kc = kb * int32_t(ROW_BYTES);
          uint32_t b_dst = sbase + S::OFF_B + stage * S::B_BYTES;
          int32_t r = trow;
          auto rows_of = [&](const CUtensorMap* map, int32_t n) {
            if constexpr (kPair)
              tma_load_2d_pair(b_dst, map, fb, kc, r);
            else
              tma_load_2d(b_dst, map, fb, kc, r);
            b_dst += uint32_t(n) * ROW_BYTES;
            r += n;
          };
          if constexpr (kPair)
            tma_load_3d_pair(sbase + S::OFF_A + stage * A_BYTES, &maps.rhs, fb, kc, wrow, t.local_group);
          else
            tma_load_3d(sbase + S::OFF_A + stage * A_BYTES, &maps.rhs, fb, kc, wrow, t.local_group);
          if (rows & 64) rows_of(&maps.lhs64, 64);
          if (rows & 32) rows_of(&maps.lhs32, 32);
          if (rows & 16) rows_of(&maps.lhs16, 16);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (kPair && lane == 0) *word(S::OFF_ISSUED) = issued;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (leader) {
      uint32_t stage = 0, phase = 0, slot = 0, slot_phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      const bool one = elected();
      const uint64_t a_desc = sw128_desc(sbase + S::OFF_A, 16, 1024), b_desc = sw128_desc(sbase + S::OFF_B, 16, 1024);
      for (int32_t item = 0; item < items && ok; ++item) {
        const GemmTile t = tile_of(item);
        const int32_t ncols = chunk_n(t);
        if (!wait_warp_cluster(acce_bar(acc), acc_phase ^ 1u, abort_flag, p.err)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * S::kChunk;
        for (int32_t kb = 0; kb < k_blocks; ++kb) {
          // Both are asked at once, by the test that does not suspend: this warp's own work for a stage is
          // as long as the stage's MMAs, and each cycle of it counts (prefill: 662 us with suspending
          // waits, 632 so, 618 with the lane elected and the descriptors made outside the loop too).
          const uint32_t turned = mbar_test_wait_cluster(turned_bar(slot), slot_phase);
          const uint32_t full = mbar_test_wait_cluster(full_bar(stage), phase);
          if (!__all_sync(0xffffffffu, turned & full) &&
              (!wait_warp_cluster(turned_bar(slot), slot_phase, abort_flag, p.err) ||
               !wait_warp(full_bar(stage), phase, abort_flag, p.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (one) {
            // a stage uses 4 blocks of a window (NVFP4) or half of them (MXFP4)
            const uint32_t sf =
                sbase + S::OFF_SF + slot * S::kParts * SF_BYTES + (kNv ? 0u : 1024u * uint32_t(kb & 1));
#pragma unroll
            for (uint32_t j = 0; j < (kNv ? 4 : 2); ++j) {
              copy_scales<kPair>(tmem_base + S::TM_SFA + 4 * j, sf + 512u * j);
              copy_scales<kPair>(tmem_base + S::TM_SFB + (kPair ? 8 : 4) * j, sf + SF_BYTES + 512u * j);
              if (kPair && ncols > 128)
                copy_scales<kPair>(tmem_base + S::TM_SFB + 8 * j + 4, sf + 2 * SF_BYTES + 512u * j);
            }
            commit<kPair>(sempty_bar(slot));  // the window is free once it is copied
            const uint64_t ad = a_desc + uint64_t(stage * (A_BYTES >> 4)), bd = b_desc + uint64_t(stage * (S::B_BYTES >> 4));
#pragma unroll
            for (uint32_t kk = 0; kk < BK / 64; ++kk) {
              const uint32_t j = kNv ? kk : kk >> 1;
              mma_fp4<kPair, kNv>(d_tmem, ad + 2 * kk, bd + 2 * kk,
                                  idesc_fp4<kNv>(S::kTileW, ncols, kNv ? 0u : 2u * (kk & 1)),
                                  tmem_base + S::TM_SFA + 4 * j, tmem_base + S::TM_SFB + (kPair ? 8 : 4) * j,
                                  (uint32_t(kb) | kk) != 0 ? 1u : 0u);
            }
            commit<kPair>(empty_bar(stage));
            if (kb == k_blocks - 1) commit<kPair>(accf_bar(acc));
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++slot == kScales) {
            slot = 0;
            slot_phase ^= 1u;
          }
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (one) {
        if constexpr (kPair)
          mma_commit_pair(done_bar, 0x1);
        else
          mma_commit(done_bar);
        drain_bar(done_bar, 0);
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- copies of scales (both CTAs)
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int32_t item = 0; item < items && ok; ++item) {
      const GemmTile t = tile_of(item);
      const int32_t wrow = t.n_tile * S::kTileW + int32_t(rank) * BW;
      const int32_t wrows = max(0, min(BW, p.n - wrow));
      const uint32_t a_bytes = uint32_t(wrows) * 16u, b_bytes = uint32_t(t.row_end - t.row0) * 16u;
      const uint8_t* a_src = p.rhs_scale + (int64_t(t.local_group) * windows * p.n + wrow) * 16;
      const uint8_t* b_src = p.lhs_scale + int64_t(t.row0) * 16;
      for (int32_t kb = 0; kb < k_blocks; ++kb) {
        if (!wait_warp(sempty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (elected()) {
          const uint32_t dst = sbase + S::OFF_SF + stage * S::kParts * SF_BYTES;
          const int64_t win = kNv ? kb : kb >> 1;
          mbar_arrive_expect_tx(sfull_bar(stage), a_bytes + b_bytes);
          if (wrows > 0) bulk_load(dst, a_src + win * p.n * 16, a_bytes, sfull_bar(stage));
          bulk_load(dst + SF_BYTES, b_src + win * p.m * 16, b_bytes, sfull_bar(stage));
        }
        __syncwarp();
        ++issued;
        if (++stage == kScales) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp > 10) {
    // ---------------------------------------------------------------- scales into the MMA's order (both CTAs)
    const int64_t stages = int64_t(items) * k_blocks;
    // A warp has stages of its own: a parity wait tells a phase from the one before it only, so
    // whoever waits on a barrier has to have seen each of its phases.
    uint32_t phase = 0, turns = 0;
    bool ok = true;
    for (int64_t i0 = 0; i0 < stages && ok; i0 += kScales, phase ^= 1u) {
      ++turns;
      for (int32_t stage = warp - 11; stage < kScales && i0 + stage < stages; stage += kTurners) {
        if (!wait_warp(sfull_bar(stage), phase, abort_flag, p.err)) {
          ok = false;
          break;
        }
        turn_scales<S::kParts>(sbase + S::OFF_SF + stage * S::kParts * SF_BYTES, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (!kPair)
            mbar_arrive(turned_bar(stage));
          else if (leader)
            mbar_arrive_expect_tx(turned_bar(stage), kSignalBytes);
          else
            signal_leader(sbase + S::OFF_SIGNAL, turned_bar(stage));
          if (kPair) word(S::OFF_TURNS)[stage] = turns;
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue (both CTAs)
    // TMEM lane = this CTA's weight row = output column; TMEM column = row of the chunk.
    const int quarter = warp & 3, set = (warp - 2) >> 2;
    const uint32_t buf = sbase + S::OFF_OUT + uint32_t(warp - 2) * OUT_BYTES;
    const uint32_t acce0 = kPair ? mapa_shared(acce_bar(0), 0) : acce_bar(0);
    uint32_t acc = 0, acc_phase = 0;
    constexpr int kBlocks = (S::kChunk / 32 + 1) / 2;  // of 32 rows, for each set
    // What a tile's outputs are scaled by, loaded a tile ahead.  bf16: this thread's weight rows are
    // lane / 4 + 8 i; f32: weight row lane (i = 0).  Row scales: block i's row `lane`.
    struct Scales {
      float ws[4], bias[4], rs[kBlocks];
    } next;
    auto col_of = [&](const GemmTile& t) { return t.n_tile * S::kTileW + int32_t(rank) * BW + quarter * 32; };
    auto load_scales = [&](const GemmTile& t, Scales& s) {
      const int64_t w0 = int64_t(t.local_group) * p.n;
#pragma unroll
      for (int i = 0; i < (kOutF32 ? 1 : 4); ++i) {
        const int32_t c = col_of(t) + (kOutF32 ? lane : lane / 4 + 8 * i);
        s.ws[i] = c < p.n && p.rhs_row_scale != nullptr ? __ldg(p.rhs_row_scale + w0 + c) : 1.f;
        s.bias[i] = c < p.n && p.bias != nullptr ? load_bias(p, w0 + c) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        const int32_t r = t.row0 + 32 * (2 * i + set) + lane;
        s.rs[i] = p.lhs_row_scale != nullptr && r < t.row_end ? __ldg(p.lhs_row_scale + r) : 1.f;
      }
    };
    GemmTile t{};
    if (items > 0) {
      t = tile_of(0);
      load_scales(t, next);
    }
    for (int32_t item = 0; item < items; ++item) {
      const int32_t rows = t.row_end - t.row0, ncols = chunk_n(t), col0 = col_of(t), row0 = t.row0;
      const Scales now = next;
      if (item + 1 < items) {
        t = tile_of(item + 1);
        load_scales(t, next);
      }
      if (!wait_warp(accf_bar(acc), acc_phase, abort_flag, p.err)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (uint32_t(quarter * 32) << 16) + acc * S::kChunk;
      // The accumulator may be overwritten: this warp's loads of it have completed (wait::ld), and
      // nothing else is handed over, so the arrive orders no memory.  (With release at cluster scope it
      // waits for the warp's stores to `out`, some 1500 cycles a tile.)
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_relaxed_cluster(acce0 + 8 * acc);
          else
            mbar_arrive(acce0 + 8 * acc);
        }
      };
      if (32 * set >= ncols) release();
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const int32_t c0 = 32 * (2 * b + set);
        if (c0 < ncols) {
          const bool last = c0 + 64 >= ncols;
          if constexpr (kOutF32) {
            uint32_t v[32];
            tmem_ld_32cols(tbase + c0, v);
            if (last) release();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float r = fmaf(__uint_as_float(v[i]) * __shfl_sync(0xffffffffu, now.rs[b], i), now.ws[0], now.bias[0]);
              if (col0 + lane < p.n && c0 + i < rows)
                static_cast<float*>(p.out)[int64_t(row0 + c0 + i) * p.n + col0 + lane] = r;
            }
          } else {
            uint32_t v[2][16];
            tmem_ld_16x32(tbase + c0, v[0]);
            tmem_ld_16x32(tbase + c0 + (16u << 16), v[1]);
            tmem_wait_ld16(v[0]);
            tmem_wait_ld16(v[1]);
            if (last) release();
            const uint32_t at = buf + uint32_t(8 * (lane >> 4) + (lane & 7)) * OUT_PITCH + uint32_t(lane >> 3 & 1) * 16u;
            const int32_t c = col0 + 8 * (lane & 3);
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + int64_t(row0 + c0) * p.n + c;
#pragma unroll
            for (int g = 0; g < 4; g += 2) {  // 16 rows at a time
              float r[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                r[i] = __shfl_sync(0xffffffffu, now.rs[b], 8 * (g + i / 2) + 2 * (lane & 3) + (i & 1));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t m[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // matrix q: rows 8 (g + q / 2) .. and columns 16 h + 8 (q & 1) ..
                  const int i = 4 * (g + q / 2) + 2 * (q & 1), f = 2 * h + (q & 1);
                  m[q] = pack_bf16x2(fmaf(__uint_as_float(v[h][i]) * r[q & 2], now.ws[f], now.bias[f]),
                                     fmaf(__uint_as_float(v[h][i + 1]) * r[(q & 2) + 1], now.ws[f], now.bias[f]));
                }
                stmatrix_trans(at + uint32_t(h) * 32u, m[0], m[1], m[2], m[3]);
              }
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int32_t w = 8 * q + (lane >> 2), row = 8 * g + w;
                const uint4 x = ld_shared_v4(buf + uint32_t(w) * OUT_PITCH + uint32_t(lane & 3) * 16u);
                if (c < p.n && c0 + row < rows) st_global_v4(o + int64_t(row) * p.n, x.x, x.y, x.z, x.w);
              }
              __syncwarp();
            }
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
    const int64_t stride = int64_t(gridDim.x) * 256;
    for (int64_t i = int64_t(blockIdx.x) * 256 + (threadIdx.x - 64); i < n_all; i += stride) {
      const int64_t byte = i < n_lo ? i * 16 : hi_begin + (i - n_lo) * 16;
      st_global_v4(static_cast<uint8_t*>(p.out) + byte, 0u, 0u, 0u, 0u);
    }
  }

  tc_fence_before();
  __syncthreads();
  // Every role has ended.  If a wait of this CTA gave up, copies may be in flight that nobody waited for, its
  // own producers' or not: the last kScales of scales, which are this CTA's affair alone, and the last kStages
  // of codes.  (Where none gave up, each copy has been waited for by the warp that it was made for.)
  const bool gave_up = *abort_flag != 0u;
  if (gave_up && warp == 10 && lane == 0) {
    for (uint32_t i = issued > kScales ? issued - kScales : 0u; i < issued; ++i)
      drain_bar(sfull_bar(i % kScales), (i / kScales) & 1u);
  }
  if constexpr (!kPair) {
    if (gave_up && warp == 0 && lane == 0) {
      for (uint32_t i = issued > kStages ? issued - kStages : 0u; i < issued; ++i)
        drain_bar(full_bar(i % kStages), (i / kStages) & 1u);
    }
  } else {
    if (leader && gave_up && threadIdx.x == 0) {
      st_shared_cluster_u32(mapa_shared(sbase + S::OFF_UNWIND, 1), 1u);
      st_shared_cluster_u32(mapa_shared(sbase + S::OFF_ABORT, 1), 1u);  // the follower's waits end too
    }
    cluster_sync();  // the roles of both CTAs have ended, the leader's MMAs are done, and both know of `unwind`
    // A follower that gave up leaves the leader's MMA warp a stage, or an accumulator that it asks for, short
    // unless that one is done, so the leader's giving up is what counts.  Then the codes of both CTAs and the
    // follower's signals are settled at the leader's barriers before either CTA may end.
    if (leader ? gave_up : *word(S::OFF_UNWIND) != 0u) {
      if (leader && threadIdx.x == 0) {
        auto peer = [&](uint32_t off) { return ld_shared_cluster_u32(mapa_shared(sbase + off, 1)); };
        // stage i of the sequence belongs to the pair's (i / k_blocks)-th item
        pair_settle<kStages>(full_bar(0), peer(S::OFF_ISSUED), issued, [&](uint32_t i) {
          return code_bytes(lane_tile(int32_t(i / uint32_t(k_blocks))));
        });
        for (uint32_t s = 0; s < kScales; ++s) {
          // The follower is a turn ahead at most: the next needs an MMA after the leader's.
          const uint32_t turns = peer(S::OFF_TURNS + 4 * s);
          if (turns > word(S::OFF_TURNS)[s]) mbar_arrive_expect_tx(turned_bar(s), kSignalBytes);
          if (turns > 0) drain_bar(turned_bar(s), (turns - 1) & 1u);
        }
      }
      cluster_sync();
    }
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair)
      tmem_dealloc_pair(tmem_base, S::kColumns);
    else
      tmem_dealloc(tmem_base, S::kColumns);
  }
}

template <bool kPair, bool kNv, bool kOutF32>
cudaError_t launch(const Maps& maps, const Params& p, int sms, cudaStream_t stream) {
  using S = Shape<kPair>;
  auto kern = gemm_fp4_kernel<kPair, kNv, kOutF32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::SMEM_BYTES));
  if (e != cudaSuccess) return e;
  unsigned grid = unsigned(kPair ? sms & ~1 : sms);
  if (kPair) {
    // One pair per co-resident cluster slot (persistent kernel).
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM_BYTES;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorLaunchOutOfResources;
    if (2 * clusters < int(grid)) grid = unsigned(2 * clusters);
  }
  return launch_dependent(kern, grid, kThreads, S::SMEM_BYTES, stream, S::kCtas, maps, p);
}

template <bool kPair>
cudaError_t launch_shape(const Maps& maps, const Params& p, bool nv, bool out_f32, int sms, cudaStream_t stream) {
  if (nv)
    return out_f32 ? launch<kPair, true, true>(maps, p, sms, stream) : launch<kPair, true, false>(maps, p, sms, stream);
  return out_f32 ? launch<kPair, false, true>(maps, p, sms, stream) : launch<kPair, false, false>(maps, p, sms, stream);
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
  if (m < 0 || m > kMaxSize || k < 32 || k > kMaxSize || k % 32 != 0 || n < 8 || n > kMaxSize || n % 8 != 0)
    return GMM_ERR_SHAPE;
  if (num_total_groups < 1 || num_total_groups > GMM_MAX_GROUPS || num_local_groups < 1 ||
      num_local_groups > num_total_groups)
    return GMM_ERR_SHAPE;
  if (group_offset < 0 || group_offset > num_total_groups - num_local_groups) return GMM_ERR_GROUP_OFFSET;
  if (((m + 31) / 32 + num_local_groups) * ((n + BW - 1) / BW) > INT32_MAX) return GMM_ERR_SHAPE;
  if (!aligned(lhs_codes, 16) || !aligned(lhs_block_scale, 16) || !aligned(rhs_codes, 16) ||
      !aligned(rhs_block_scale, 16) || !aligned(out, 16) || !aligned(lhs_row_scale, 4) || !aligned(rhs_row_scale, 4) ||
      !aligned(rhs_bias, bias_dtype == GMM_DTYPE_F32 ? 4 : 2) || !aligned(group_sizes, 4))
    return GMM_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < GMM_WORKSPACE_MIN_BYTES || !aligned(workspace, 16))
    return GMM_ERR_WORKSPACE;
  int sms = 0;
  if (int st = require_device(&sms)) return st;
  if (m == 0) return GMM_OK;
  // One SM up to 16 rows a group on average, pairs above.  With equal groups the two meet at 32 rows (64
  // experts, 4096 -> 2048: 4 rows 53 us against the pairs' 55, 32 rows 55 both, 64 rows 74 against 57;
  // 8 experts: 14 against 16, 14 against 16, 18 against 16), but where the average is over 16 some groups
  // are well over 32, for which one SM's tile meets its weights again for every 32 rows.
  const bool pair = m >= int64_t(16) * num_total_groups;
  Maps maps;
  for (const auto& [map, rows] : {std::pair<CUtensorMap*, uint32_t>(&maps.lhs64, 64u), {&maps.lhs32, 32u},
                                  {&maps.lhs16, 16u}}) {
    const uint64_t dims[2] = {uint64_t(k / 2), uint64_t(m)};
    const uint32_t box[2] = {BK / 2, rows};
    if (int st = byte_map(map, 2, lhs_codes, dims, box)) return st;
  }
  {
    const uint64_t dims[3] = {uint64_t(k / 2), uint64_t(n), uint64_t(num_local_groups)};
    const uint32_t box[3] = {BK / 2, BW, 1};
    if (int st = byte_map(&maps.rhs, 3, rhs_codes, dims, box)) return st;
  }
  const Params p{group_sizes, num_total_groups, group_offset, num_local_groups, int32_t(m), int32_t(n), int32_t(k),
                 static_cast<const uint8_t*>(lhs_block_scale), static_cast<const uint8_t*>(rhs_block_scale),
                 lhs_row_scale, rhs_row_scale, out, rhs_bias, bias_dtype == GMM_DTYPE_F32 ? 1 : 0,
                 static_cast<uint32_t*>(workspace)};
  if (call_log_enabled())
    std::fprintf(stderr, "libgmm: gmm_fp4 m=%lld k=%lld n=%lld groups=%d local=%d offset=%d format=%s out=%s kernel=%s\n",
                 (long long)m, (long long)k, (long long)n, num_total_groups, num_local_groups, group_offset,
                 nv ? "nvfp4" : "mxfp4", out_dtype == GMM_DTYPE_F32 ? "f32" : "bf16",
                 pair ? "pair" : "single");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = out_dtype == GMM_DTYPE_F32;
  const cudaError_t e = pair ? launch_shape<true>(maps, p, nv, f32, sms, s) : launch_shape<false>(maps, p, nv, f32, sms, s);
  return e == cudaSuccess ? GMM_OK : record_cuda_error(e);
}
