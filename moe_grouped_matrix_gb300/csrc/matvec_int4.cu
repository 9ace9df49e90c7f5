// Products of few tokens with 4-bit integer weights in groups of 32, 64 or 128 k:
//   h[t, j] = sum over groups of scale * sum of (code - zero) x
// for the expert of each slot (t, j), in the order of the tokens.
//
// Bound by memory: half a byte a weight, read once.  At 6.8 TB/s an SM gets some 47
// weights a cycle, and may spend 2.7 issue slots of a lane on each; one fp32
// multiply-add with its conversion takes about 2 for a single token.  So the sums run on
// mma.sync m16n8k16, 16 weight rows by 8 columns: the codes become bf16 in 1.4
// instructions each for all 8 columns (a nibble or-ed into 128's mantissa is 128 + code,
// and one packed subtraction takes 128 and the zero point off, exactly), x is bf16 as it
// stands, products are exact and sums fp32.  A group's sum is scaled in fp32.  A matrix
// instruction's k are a set without an order, so a lane takes the eight k of a 32-bit
// word for its own, and x is permuted alike.
//
// A warp streams windows of 16 rows by 256 k through a ring of its own in shared memory,
// by asynchronous copies that only it waits for: no barrier between warps but one for each
// unit's sums.  Whole 128-byte lines of each row are copied, 16-byte chunks permuted by row
// so that reading a chunk's word by 8 rows and 4 lanes meets all banks.
//
// A unit is 8 / KW tiles of 16 rows (with an activation 8 gates and the 8 rows they gate),
// KW warps to a tile along k, for
//   - up to 8 slots of one expert, or
//   - with weights, 8 tokens: all of their experts, one after another, columns the
//     tokens, so that the sum over a token's slots stays in registers.
#include <cuda_bf16.h>

#include <climits>

#include "activation.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kWindow = 256;                 // k of a stage
constexpr int kCols = 8;                     // columns of an item
constexpr int kMaxSlots = 512;               // slots of a launch
constexpr int kCodeBytes = 16 * kWindow / 2;

struct Params {
  const __nv_bfloat16* x;
  int64_t x_token, x_slot;  // elements between tokens, and between a token's slots
  const uint8_t* codes;
  const uint8_t* scale;  // bf16, by windows
  const uint8_t* zero;
  int32_t experts, n, k, windows, tiles;  // tiles of 16 rows of an expert
  const int32_t* chosen;  // NULL: expert 0
  int32_t tokens, topk;
  const float* weights;   // NULL: no sum over slots
  int32_t act;            // of gated tiles
  void* out;
  int32_t out_n, out_f32;  // columns of out, its type
  int32_t kw;             // warps to a tile: 2, 4 or 8
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  const int bytes = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two codes, at bits 0-3 and 16-19 of w, as bf16 with `off` = 128 + zero taken off.
template <bool kZero>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, __nv_bfloat162 off) {
  // two's complement + 8 is the code with its top bit flipped
  const uint32_t raw = (w & 0x000F000Fu) ^ (kZero ? 0x43004300u : 0x43084308u);
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&raw), off);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kGroup, bool kZero>
struct Stage {
  static constexpr int kEach = kWindow / kGroup;
  static constexpr int kScale = kCodeBytes, kZeros = kScale + 16 * kEach * 2;
  static constexpr int kBytes = kZeros + (kZero ? 16 * kEach : 0);
};

// The table of items that each CTA makes of the slots.
struct Table {
  int32_t expert[kMaxSlots];          // of each slot; then of each item
  int16_t slot[kMaxSlots][kCols];     // of each item's columns; -1: none
  int16_t first[kMaxSlots / kCols + kMaxSlots + 1];  // with weights: first item of each 8 tokens
  int32_t items;
  int32_t warp_heads[kWarps];
};

// Where a warp is in its sequence of (unit, pair of item and window).
struct Place {
  int64_t unit;
  int32_t pair, end;       // of the warp in the unit
  int32_t item, window;
  int64_t half0, half1;    // expert * n + first row of each half tile; half1 < 0: none
};

template <int kGroup, bool kZero, bool kGated, bool kSum, int kStages>
__global__ void __launch_bounds__(kThreads, 2) matvec_kernel(Params p) {
  using S = Stage<kGroup, kZero>;
  griddep_begin();
  p.x = after_begin(p.x), p.codes = after_begin(p.codes), p.scale = after_begin(p.scale);
  p.zero = after_begin(p.zero), p.chosen = after_begin(p.chosen), p.weights = after_begin(p.weights);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Table table;
  __shared__ float part[2][kWarps][16][kCols + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slots = p.tokens * p.topk;
  const int KW = p.kw, kTiles = kWarps / KW;  // tiles of a unit

  // ---- items: slots of the same expert in their order, 8 at a time (kSum: those of 8 tokens; a
  // token's second slot of the same expert has an item of its own).  A head is an item's first slot.
  for (int i = tid; i < slots; i += kThreads) {
    const int e = p.chosen != nullptr ? p.chosen[i] : 0;
    table.expert[i] = e >= 0 && e < p.experts ? e : -1;
  }
  for (int i = tid; i < kMaxSlots * kCols / 2; i += kThreads) reinterpret_cast<uint32_t*>(table.slot)[i] = 0xFFFFFFFFu;
  if (tid == 0) table.items = 0;
  __syncthreads();
  // a slot's item: its head's, of which this thread keeps what it needs until all have read the table
  int head[kMaxSlots / kThreads], column[kMaxSlots / kThreads], mine[kMaxSlots / kThreads];
#pragma unroll
  for (int r = 0; r < kMaxSlots / kThreads; ++r) {
    const int i = r * kThreads + tid;
    head[r] = -1, column[r] = 0, mine[r] = -1;
    if (i >= slots) continue;
    const int e = table.expert[i];
    mine[r] = e;
    if (e < 0) continue;
    head[r] = i;
    if constexpr (kSum) {
      const int t = i / p.topk, t0 = t / kCols * kCols;
      column[r] = t - t0;
      int twin = 0;  // earlier slots of the token with this expert
      for (int j = t * p.topk; j < i; ++j) twin += table.expert[j] == e;
      // the first token of the eight with so many of them
      for (int u = t0; u < t; ++u) {
        int seen = 0, at = -1;
        for (int j = u * p.topk; j < (u + 1) * p.topk; ++j)
          if (table.expert[j] == e && seen++ == twin) at = j;
        if (at >= 0) {
          head[r] = at;
          break;
        }
      }
    } else {
      int before = 0, at = i;
      for (int j = 0; j < i; ++j)
        if (table.expert[j] == e) {
          if (before % kCols == 0) at = j;
          ++before;
        }
      column[r] = before % kCols;
      head[r] = column[r] == 0 ? i : at;
    }
  }
  __syncthreads();
  // heads numbered in the order of their slots: expert[] turns into that of the items, and a head's
  // number goes to number[] (the ring, not yet in use)
  int32_t* number = reinterpret_cast<int32_t*>(smem);
#pragma unroll
  for (int r = 0; r < kMaxSlots / kThreads; ++r) {
    const int i = r * kThreads + tid;
    const bool is_head = head[r] == i && mine[r] >= 0;
    const uint32_t ballot = __ballot_sync(0xffffffffu, is_head);
    if (lane == 0) table.warp_heads[warp] = __popc(ballot);
    __syncthreads();
    int at = table.items;
    for (int w = 0; w < warp; ++w) at += table.warp_heads[w];
    at += __popc(ballot & ((1u << lane) - 1u));
    if constexpr (kSum) {
      if (i < slots && i % (kCols * p.topk) == 0) table.first[i / (kCols * p.topk)] = int16_t(at);
    }
    if (is_head) number[i] = at, table.expert[at] = mine[r];  // at <= i: read above by all
    __syncthreads();
    if (tid == 0)
      for (int w = 0; w < kWarps; ++w) table.items += table.warp_heads[w];
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kMaxSlots / kThreads; ++r)
    if (head[r] >= 0) table.slot[number[head[r]]][column[r]] = int16_t(r * kThreads + tid);
  const int chunks = (p.tokens + kCols - 1) / kCols;
  if (kSum && tid == 0) table.first[chunks] = int16_t(table.items);
  __syncthreads();

  auto put = [&](int64_t row, int64_t c, float v) {
    if (p.out_f32 != 0)
      static_cast<float*>(p.out)[row * p.out_n + c] = v;
    else
      static_cast<__nv_bfloat16*>(p.out)[row * p.out_n + c] = __float2bfloat16_rn(v);
  };
  if constexpr (!kSum) {  // rows of slots without an expert
#pragma unroll
    for (int r = 0; r < kMaxSlots / kThreads; ++r) {
      uint32_t none = __ballot_sync(0xffffffffu, r * kThreads + tid < slots && mine[r] < 0);
      while (none != 0) {
        const int64_t i = r * kThreads + warp * 32 + __ffs(none) - 1;
        none &= none - 1;
        for (int64_t c = int64_t(blockIdx.x) * 32 + lane; c < p.out_n; c += int64_t(gridDim.x) * 32) put(i, c, 0.f);
      }
    }
  }

  // ---- the warp's sequence
  const int tile_units = (p.tiles + kTiles - 1) / kTiles;
  const int64_t units = int64_t(kSum ? chunks : table.items) * tile_units;
  const int kw = warp % KW;
  const uint32_t ring = smem_u32(smem) + uint32_t(warp) * (kStages * S::kBytes);

  auto halves = [&](Place& at) {  // of the tile, in the item's expert
    const int tile = int(at.unit % tile_units) * kTiles + warp / KW;
    const int64_t base = int64_t(table.expert[at.item]) * p.n;
    if constexpr (kGated) {
      at.half0 = base + tile * 8, at.half1 = base + p.n / 2 + tile * 8;
    } else {
      at.half0 = base + tile * 16, at.half1 = tile * 16 + 8 < p.n ? base + tile * 16 + 8 : -1;
    }
  };
  // The first pair of a unit, or of the next that has any for this warp.
  auto enter = [&](Place& at) {
    for (; at.unit < units; at.unit += gridDim.x) {
      const int group = int(at.unit / tile_units), tile = int(at.unit % tile_units) * kTiles + warp / KW;
      const int first = kSum ? table.first[group] : group, n = kSum ? table.first[group + 1] - first : 1;
      const int pairs = tile < p.tiles ? n * p.windows : 0;
      at.pair = int(int64_t(pairs) * kw / KW), at.end = int(int64_t(pairs) * (kw + 1) / KW);
      if (at.pair < at.end) {
        at.item = first + at.pair / p.windows, at.window = at.pair % p.windows;
        halves(at);
        return;
      }
    }
  };
  auto next = [&](Place& at) {
    if (++at.pair == at.end) {
      at.unit += gridDim.x;
      enter(at);
    } else if (++at.window == p.windows) {
      at.window = 0, ++at.item;
      halves(at);
    }
  };
  auto fetch = [&](const Place& at, int stage) {
    const uint32_t to = ring + uint32_t(stage) * S::kBytes;
    const int chunk = lane & 7;
    const bool in = at.window * kWindow + chunk * 32 < p.k;
    const int64_t pitch = p.k / 2, off = int64_t(at.window) * (kWindow / 2) + (in ? chunk * 16 : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = i * 4 + (lane >> 3);
      const bool there = in && (i < 2 || at.half1 >= 0);
      const int64_t r = (i < 2 || at.half1 < 0 ? at.half0 : at.half1) + (row & 7);
      copy16(to + row * 128 + ((chunk ^ (row & 7)) << 4), p.codes + r * pitch + off, there);
    }
    // scales and zero points: 8 rows' are contiguous.  half = (expert, row) -> (expert, window, row)
    auto at_window = [&](int64_t half) {
      const int64_t e = table.expert[at.item];
      return (e * p.windows + at.window) * p.n + (half - e * p.n);
    };
    constexpr int kHalf = 8 * S::kEach;  // values of half a tile
    const int which = lane / (kHalf / 8), piece = lane % (kHalf / 8);
    if (which < 2) {
      const int64_t half = which == 0 || at.half1 < 0 ? at.half0 : at.half1;
      copy16(to + S::kScale + which * kHalf * 2 + piece * 16, p.scale + at_window(half) * (S::kEach * 2) + piece * 16,
             which == 0 || at.half1 >= 0);
    }
    if constexpr (kZero) {
      const int whichz = lane / (kHalf / 16), piecez = lane % (kHalf / 16);
      if (whichz < 2) {
        const int64_t half = whichz == 0 || at.half1 < 0 ? at.half0 : at.half1;
        copy16(to + S::kZeros + whichz * kHalf + piecez * 16, p.zero + at_window(half) * S::kEach + piecez * 16,
               whichz == 0 || at.half1 >= 0);
      }
    }
  };

  const int g = lane >> 2, t4 = lane & 3;
  Place ahead, here;
  ahead.unit = blockIdx.x;
  enter(ahead);
  here = ahead;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (ahead.unit < units) {
      fetch(ahead, s);
      next(ahead);
    }
    copies_commit();
  }
  int stage = 0, parity = 0;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x, parity ^= 1) {
    float res[4] = {0.f, 0.f, 0.f, 0.f};
    int item = -1;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const __nv_bfloat16* xp = nullptr;  // column g of the item
    float w0 = 1.f, w1 = 1.f;           // weights of columns 2 t4 and 2 t4 + 1
    auto flush = [&] {
      res[0] += w0 * acc[0], res[1] += w1 * acc[1], res[2] += w0 * acc[2], res[3] += w1 * acc[3];
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    };
    while (here.unit == unit) {
      if (here.item != item) {
        if (kSum && item >= 0) flush();
        item = here.item;
        const int s = table.slot[item][g];
        xp = s < 0 ? nullptr : p.x + (s / p.topk) * p.x_token + (s % p.topk) * p.x_slot;
        if constexpr (kSum) {
          const int s0 = table.slot[item][2 * t4], s1 = table.slot[item][2 * t4 + 1];
          w0 = s0 < 0 ? 0.f : p.weights[s0], w1 = s1 < 0 ? 0.f : p.weights[s1];
        }
      }
      // x of this window for all groups
      const int k0 = here.window * kWindow;
      const int groups = min(S::kEach, (p.k - k0) / kGroup);
      copies_wait<kStages - 2>();
      __syncwarp();
      if (ahead.unit < units) {
        fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
        next(ahead);
      }
      copies_commit();
      const uint32_t at = ring + uint32_t(stage) * S::kBytes;
#pragma unroll
      for (int q = 0; q < S::kEach; ++q) {
        if (q < groups) {
          float c[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t z0 = 8, z1 = 8;
          if constexpr (kZero) {
            z0 = smem[at - smem_u32(smem) + S::kZeros + g * S::kEach + q];
            z1 = smem[at - smem_u32(smem) + S::kZeros + (g + 8) * S::kEach + q];
          }
          const uint32_t o0 = 0x43004300u + z0 * 0x00010001u, o1 = 0x43004300u + z1 * 0x00010001u;
          const __nv_bfloat162 off0 = *reinterpret_cast<const __nv_bfloat162*>(&o0);
          const __nv_bfloat162 off1 = *reinterpret_cast<const __nv_bfloat162*>(&o1);
#pragma unroll
          for (int j = 0; j < kGroup / 32; ++j) {
            const int chunk = q * (kGroup / 32) + j;
            uint4 b = make_uint4(0, 0, 0, 0);
            if (xp != nullptr) b = __ldg(reinterpret_cast<const uint4*>(xp + k0 + chunk * 32 + t4 * 8));
            const uint32_t wa = lds32(at + g * 128 + ((chunk ^ g) << 4) + t4 * 4);
            const uint32_t wb = lds32(at + (g + 8) * 128 + ((chunk ^ g) << 4) + t4 * 4);
            mma(c, two_codes<kZero>(wa, off0), two_codes<kZero>(wb, off1), two_codes<kZero>(wa >> 4, off0),
                two_codes<kZero>(wb >> 4, off1), __byte_perm(b.x, b.z, 0x5410), __byte_perm(b.x, b.z, 0x7632));
            mma(c, two_codes<kZero>(wa >> 8, off0), two_codes<kZero>(wb >> 8, off1), two_codes<kZero>(wa >> 12, off0),
                two_codes<kZero>(wb >> 12, off1), __byte_perm(b.y, b.w, 0x5410), __byte_perm(b.y, b.w, 0x7632));
          }
          const __nv_bfloat16* sc = reinterpret_cast<const __nv_bfloat16*>(smem + (at - smem_u32(smem)) + S::kScale);
          const float s0 = __bfloat162float(sc[g * S::kEach + q]), s1 = __bfloat162float(sc[(g + 8) * S::kEach + q]);
          acc[0] = fmaf(s0, c[0], acc[0]), acc[1] = fmaf(s0, c[1], acc[1]);
          acc[2] = fmaf(s1, c[2], acc[2]), acc[3] = fmaf(s1, c[3], acc[3]);
        }
      }
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
      next(here);
    }
    flush();
    part[parity][warp][g][2 * t4] = res[0], part[parity][warp][g][2 * t4 + 1] = res[1];
    part[parity][warp][g + 8][2 * t4] = res[2], part[parity][warp][g + 8][2 * t4 + 1] = res[3];
    __syncthreads();
    // sums over the warps of a tile, and out
    const int group = int(unit / tile_units), tile0 = int(unit % tile_units) * kTiles;
    constexpr int kRows = kGated ? 8 : 16;
    for (int i = tid; i < kTiles * kRows * kCols; i += kThreads) {
      const int row = i % kRows, tile = i / kRows % kTiles, col = i / (kRows * kTiles);
      int64_t to;
      if constexpr (kSum) {
        const int t = group * kCols + col;
        if (t >= p.tokens) continue;
        to = t;
      } else {
        to = table.slot[group][col];
        if (to < 0) continue;
      }
      const int c = (tile0 + tile) * kRows + row;
      if (c >= p.out_n) continue;
      float v = 0.f;
      for (int w = 0; w < KW; ++w) v += part[parity][tile * KW + w][row][col];
      if constexpr (kGated) {
        float u = 0.f;
        for (int w = 0; w < KW; ++w) u += part[parity][tile * KW + w][row + 8][col];
        v = (p.act == GMM_ACT_SILU ? act_value<GMM_ACT_SILU>(v) : act_value<GMM_ACT_GELU>(v)) * u;
      }
      put(to, c, v);
    }
  }
  copies_wait<0>();
}

template <int kGroup, bool kZero, bool kGated, bool kSum>
cudaError_t launch(const Params& p, int64_t units, int sms, cudaStream_t stream) {
  // two CTAs to an SM: 114 KB each, 21 of them the table and the sums
  constexpr int kStages = 94000 / (kWarps * Stage<kGroup, kZero>::kBytes);
  constexpr size_t smem = size_t(kWarps) * kStages * Stage<kGroup, kZero>::kBytes;
  auto kern = matvec_kernel<kGroup, kZero, kGated, kSum, kStages>;
  // set for every launch: the attribute is the current device's
  if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem))) return e;
  const int64_t grid = units < 2 * sms ? units : 2 * sms;
  return launch_dependent(kern, unsigned(grid < 1 ? 1 : grid), kThreads, smem, stream, 1, p);
}

template <int kGroup, bool kZero>
cudaError_t by_form(const Params& p, int64_t units, int sms, cudaStream_t stream) {
  if (p.weights != nullptr) return launch<kGroup, kZero, false, true>(p, units, sms, stream);
  return p.act != GMM_ACT_NONE ? launch<kGroup, kZero, true, false>(p, units, sms, stream)
                               : launch<kGroup, kZero, false, false>(p, units, sms, stream);
}

cudaError_t matvec(Params p, int group, int sms, cudaStream_t stream) {
  p.kw = p.windows >= 8 ? 8 : p.windows >= 4 || p.weights != nullptr ? 4 : 2;
  // units at most: an item for each slot, or 8 tokens
  const int64_t groups = p.weights != nullptr ? (p.tokens + kCols - 1) / kCols : int64_t(p.tokens) * p.topk;
  const int64_t units = groups * ((p.tiles + kWarps / p.kw - 1) / (kWarps / p.kw));
  const bool zero = p.zero != nullptr;
  switch (group) {
    case 32: return zero ? by_form<32, true>(p, units, sms, stream) : by_form<32, false>(p, units, sms, stream);
    case 64: return zero ? by_form<64, true>(p, units, sms, stream) : by_form<64, false>(p, units, sms, stream);
    default: return zero ? by_form<128, true>(p, units, sms, stream) : by_form<128, false>(p, units, sms, stream);
  }
}

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace gmmk

extern "C" int gmm_matvec_int4(const void* x, int64_t tokens, int64_t k, int64_t x_ld, int x_per_slot, const void* codes,
                               const void* scale, const void* zero, int32_t group, int32_t num_experts, int64_t n,
                               const int32_t* experts, int32_t topk, const float* weights, int act, void* out,
                               int out_dtype, void* stream) {
  using namespace gmmk;
  if (out_dtype != GMM_DTYPE_BF16 && out_dtype != GMM_DTYPE_F32) return GMM_ERR_DTYPE;
  if (tokens < 0 || tokens > kMaxSize || k < 1 || k > kMaxSize || n < 1 || n > kMaxSize || n % 8 != 0 ||
      (group != 32 && group != 64 && group != 128) || k % group != 0 || num_experts < 1 ||
      num_experts > GMM_MAX_GROUPS || topk < 1 || topk > GMM_MAX_TOPK || (tokens > 0 && experts == nullptr && topk != 1) ||
      (act != GMM_ACT_NONE && act != GMM_ACT_SILU && act != GMM_ACT_GELU))
    return GMM_ERR_SHAPE;
  if (act != GMM_ACT_NONE && (n % 16 != 0 || weights != nullptr)) return GMM_ERR_SHAPE;
  if (x_per_slot != 0 ? false : x_ld < k || x_ld % 8 != 0) return GMM_ERR_SHAPE;
  if (tokens > 0 && (x == nullptr || codes == nullptr || scale == nullptr || out == nullptr)) return GMM_ERR_NULL;
  if (misaligned(x, 16) || misaligned(codes, 16) || misaligned(scale, 16) || misaligned(zero, 16) ||
      misaligned(experts, 4) || misaligned(weights, 4) || misaligned(out, out_dtype == GMM_DTYPE_F32 ? 4 : 2))
    return GMM_ERR_ALIGN;
  int sms = 0;
  if (int st = require_device(&sms)) return st;
  const int64_t out_n = act != GMM_ACT_NONE ? n / 2 : n;
  const int64_t most = kMaxSlots / topk / kCols * kCols;  // tokens of a launch
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t count = tokens - t0 < most ? tokens - t0 : most;
    Params p{};
    p.x_token = x_per_slot != 0 ? k * topk : x_ld, p.x_slot = x_per_slot != 0 ? k : 0;
    p.x = static_cast<const __nv_bfloat16*>(x) + t0 * p.x_token;
    p.codes = static_cast<const uint8_t*>(codes), p.scale = static_cast<const uint8_t*>(scale);
    p.zero = static_cast<const uint8_t*>(zero);
    p.experts = num_experts, p.n = int32_t(n), p.k = int32_t(k), p.windows = int32_t((k + kWindow - 1) / kWindow);
    p.tiles = int32_t((n + 15) / 16);
    p.chosen = experts == nullptr ? nullptr : experts + t0 * topk;
    p.tokens = int32_t(count), p.topk = topk;
    p.weights = weights == nullptr ? nullptr : weights + t0 * topk;
    p.act = act, p.out_n = int32_t(out_n), p.out_f32 = out_dtype == GMM_DTYPE_F32;
    const int64_t first = t0 * (weights != nullptr ? 1 : topk) * out_n;
    p.out = static_cast<char*>(out) + first * (out_dtype == GMM_DTYPE_F32 ? 4 : 2);
    const cudaError_t e = matvec(p, group, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  return GMM_OK;
}
