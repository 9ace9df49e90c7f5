// Products of few tokens with 4-bit integer weights in groups of 32, 64 or 128 k:
//   h[t, j] = sum over groups of scale * sum of (code - zero) x
// for the expert of each slot (t, j), in the order of the tokens.
//
// Bound by memory: half a byte a weight, read once.  At 6.8 TB/s an SM gets some 47 weights a cycle and
// may spend 2.7 issue slots of a lane on each; one fp32 multiply-add with its conversion takes about 2 for a
// single token.  So the sums run on mma.sync m16n8k16, 16 weight rows by 8 columns (tcgen05 wants its
// operands written to shared memory in 8 or 16 bits first, four times the bytes, for 128 rows at least).
// A bit pattern below 256 is, read as bf16, that whole number times 2^-133 (subnormals, and the first binade
// above them, whose spacing is the same), so a mask takes two codes out of a word, at its bits 0-3 and 16-19 or,
// 16 times as large, at 4-7 and 20-23, and one packed multiply-add makes both 2^-110 (code - zero), exactly
// (two's complement codes have their top bit flipped, which adds 8, and 8 is their zero point): nine
// instructions for eight weights and all their columns.
//
// Both halves of that are for the sums' precision.  Codes from 0 up, their zero points taken off through sums of
// x, took five instructions, and with a channel of x 1000 times the others that meets weights of 0 the result
// was off by up to 5e-6 of its size; it is by 1e-7, as in fp32 products.  And codes left subnormal had the matrix
// instruction cut its sums off at 2^-17 of their largest term, as it lines products up by their operands'
// exponents, which say 2^-126 for all subnormals.  1 token, 2 of 8 experts of 28672 x 4096: groups of 128 25.5 us
// for 23.0 without either, of 32 26.3 for 26.2.
//
// The other operand is x times a power of two that brings each row's largest value to between 2^90 and 2^92.
// Products are exact, sums fp32, whose least number is then at most 2^-129 of the row's largest |x|: terms
// below 2^-105 of it lose bits, before or after their scale.  A row with an infinity or NaN gives NaN, by the
// factor that takes its results to their size.  A group's sum is scaled in fp32, and the power of two taken off
// the result.  A matrix instruction's k are a set without an order, so a lane takes the eight k of a 32-bit
// word for its own, and x is permuted alike.
//
// A warp streams spans of 16 rows by 512 k through two stages of its own in shared memory, by asynchronous
// copies that only it waits for, whole lines of each row.  Teams of 1 to 16 warps share a tile along k: few
// for long streams, many for few tiles; each CTA finds the number with which the last team ends first (fixed
// at 1, 2, 4, 8, 16: 2 of 8 experts of 28672 x 4096 take 25.5, 25.0, 26.9, 30.8, 52 us for 25.4, their way back
// 46, 27, 21.7, 21.0, 22.7 for 21.3).  A unit of a team's work is a tile of 16 rows (with an activation 8 gates
// and the 8 rows they gate) for
//   - up to 8 slots of one expert, or
//   - with weights, 8 tokens: all of their experts, one after another, columns the tokens, so that the sum
//     over a token's slots stays in registers.
//
// x has to come from shared memory: through the caches a span's 8 KB for 8 columns is twice the weights'.
// Each CTA makes it ready there where it fits as a whole (2 of 8 experts of 4096 x 4096: 1 token 8.1 us for
// 8.5, 7 tokens 19.1 for 22.3; of 512 x 1024, 4 tokens 4.8 for 6.2; but 32 tokens, 4 of 16 experts of 1024 x 1024,
// 13.3 for 11.3); else a kernel ahead does, and a CTA copies one item's at a time, or where it has little to do
// reads it through the caches all the same.
//
// Measured: 1 token, 2 of 8 experts, 28672 x 4096, groups of 128, activation: 25.4 us, 121 MB at 4.8 TB/s (the
// copies alone: 21.4 us; 3.9 before the first product), instructions in 58 % of the issue slots, which wait for
// their pipes more than for memory; their way back, 4096 x 14336: 21.3 us, of which 7 before the first product,
// and 256 tiles on 152 SMs; 8 of 128 experts, 2048 x 2048, groups of 32: 8.4 us for 19 MB, 3.9 of them before the
// first product; 32 tokens, 4 of 64 experts, 2048 x 4096: 54 us for 193 MB, 3.6 TB/s.
// Of several tokens the sums over the slots read an expert's weights once for every 8 tokens: 32 tokens, 2 of 8
// experts of 4096 x 14336 take 195 us, without the sum 104.
#include <cuda_bf16.h>

#include <climits>
#include <type_traits>

#include "activation.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmmk {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kWindow = 256;                 // k of a window of scales
constexpr int kSpan = 2 * kWindow;           // k of a stage
constexpr int kCols = 8;                     // columns of an item
constexpr int kMaxSlots = 256;               // slots of a launch
constexpr int kPitch = kSpan / 2 + 16;       // bytes between rows of codes in shared memory: see below

struct Params {
  const __nv_bfloat16* x;
  int64_t x_token, x_slot;  // elements between tokens, and between a token's slots
  const uint8_t* codes;
  const uint8_t* scale;  // bf16, by windows
  const uint8_t* zero;
  int32_t experts, n, k, windows, spans, tiles;  // tiles of 16 rows of an expert
  const int32_t* chosen;  // NULL: expert 0
  int32_t tokens, topk;
  const float* weights;   // NULL: no sum over slots
  int32_t act;            // of gated tiles
  void* out;
  int32_t out_n, out_f32;  // columns of out, its type
  int32_t x_rows, x_pitch;  // rows of x made ready, and elements between them
  int32_t item_columns, item_pitch;  // kItems: most columns of an item, elements between them in shared memory
  // where not in shared memory: the rows, and what takes their results to their size
  __nv_bfloat16* ready;
  float* roots;
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  const int bytes = there ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// (v & mask) ^ flip in one instruction, which takes at most one immediate: both are kept in registers.
__device__ __forceinline__ uint32_t masked(uint32_t v, uint32_t mask, uint32_t flip) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(v), "r"(mask), "r"(flip));
  return r;
}
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
  asm volatile("" : "+r"(v));
  return v;
}
// a b + c of two bf16 each; a subnormal is taken as it is.
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// c += A B, or c = A B.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, bool first) {
  if (first)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kTop = 91;         // rows' largest values are brought to between 2^90 and 2^92
constexpr int kNotFinite = 129;  // in the place of the power of a row with an infinity or NaN

// Rows of x are made ready by windows, a warp each, 8 values a lane (zeros past k).
__device__ __forceinline__ uint4 window_of(const __nv_bfloat16* x, int k, int window) {
  const int c = window * kWindow + (threadIdx.x & 31) * 8;
  return c < k ? __ldg(reinterpret_cast<const uint4*>(x + c)) : make_uint4(0, 0, 0, 0);
}
// The largest magnitude of a lane's values, as its bits: infinities and NaN above the numbers.
__device__ __forceinline__ uint32_t largest(const uint4& v) {
  const uint32_t a = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), b = __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
  const uint32_t m = __vmaxu2(a, b);
  return max(m & 0xFFFFu, m >> 16);
}
// The power of two that a row's largest value, of these n, has or, if that is even, the next.
__device__ __forceinline__ int power_of(const uint32_t* tops, int n) {
  uint32_t top = 0;
  for (int i = threadIdx.x & 31; i < n; i += 32) top = max(top, tops[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  if (top >= 0x7F80u) return kNotFinite;
  return (top == 0 ? 0 : top < 0x80u ? 31 - __clz(int(top)) - 133 : int(top >> 7) - 127) | 1;
}
// The root of what takes a result to its own size: 2^(110 - kTop + power), or NaN.
__device__ __forceinline__ float root_of(int power) {
  return __int_as_float(power == kNotFinite ? 0x7FC00000 : (127 + (110 - kTop + power) / 2) << 23);
}
// A window of the row: x 2^(kTop - power) as bf16, in each 8 in the order of the masks, 0 4 1 5 2 6 3 7.
__device__ __forceinline__ void make_ready(const uint4& v, int k, int window, int power, __nv_bfloat16* to) {
  const int c = window * kWindow + (threadIdx.x & 31) * 8;
  if (c >= k) return;
  const int up = kTop - power, first = up / 2;  // up to 224: in two steps, each exact
  const float u0 = __int_as_float((127 + first) << 23), u1 = __int_as_float((127 + up - first) << 23);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16) * u0 * u1;
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = __float_as_uint(f[i]) >> 16 | (__float_as_uint(f[i + 4]) & 0xFFFF0000u);
  *reinterpret_cast<uint4*>(to + c) = make_uint4(out[0], out[1], out[2], out[3]);
}

// A warp's two stages: codes, scales, zero points of a span.  Rows of codes are a 16-byte piece apart
// from whole lines of banks, so that one word of 8 rows by 4 lanes meets all banks.  One stage of each
// warp on its way is 64 KB for an SM, over the 45 that memory's latency asks for at its rate.
template <int kGroup, bool kZero>
struct Ring {
  static constexpr int kEach = kWindow / kGroup;  // groups of a window
  static constexpr int kScaleAt = 16 * kPitch, kZeroAt = kScaleAt + 2 * 16 * kEach * 2;
  static constexpr int kStage = kZeroAt + (kZero ? 2 * 16 * kEach : 0);
  static constexpr int kBytes = 2 * kStage;
};

// The table of items that each CTA makes of the slots.
struct Table {
  int32_t expert[kMaxSlots];          // of each slot; -1: none
  int32_t item[kMaxSlots];            // the expert of each item
  int16_t slot[kMaxSlots][kCols];     // of each item's columns; -1: none
  int16_t head[kMaxSlots];            // of each item: its first slot
  int16_t row[kMaxSlots];             // of each slot: its row of x
  int16_t power[kMaxSlots];           // of each row of x, where they are made ready here
  int32_t columns[kMaxSlots];         // of each item
  int16_t first[kMaxSlots / kCols + kMaxSlots + 1];  // with weights: first item of each 8 tokens
  int16_t number[kMaxSlots];          // of the item that a slot is the head of
  int32_t warp_heads[kWarps];
};

// A team's place among the units: a group of items (one, or with weights those of 8 tokens) and a tile.
struct Unit {
  int32_t group, tile;
  // on by dgroup * tiles + dtile units
  __device__ __forceinline__ void advance(int dgroup, int dtile, int tiles) {
    group += dgroup, tile += dtile;
    if (tile >= tiles) tile -= tiles, ++group;
  }
};

template <bool kShared, class T>
__device__ __forceinline__ T load(const T* p) {
  if constexpr (kShared)
    return *p;
  else
    return __ldg(p);
}

// Where x comes from.
enum Mode {
  kCaches,  // rows that a kernel ahead has made ready, through the caches
  kAll,     // all rows, made ready by each CTA in its shared memory
  kItems    // such rows again, those of one item at a time copied to a CTA's shared memory
};

template <int kGroup, bool kZero, bool kGated, bool kSum, Mode kMode>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(Params p) {
  constexpr bool kStaged = kMode == kAll, kShared = kMode != kCaches;
  static_assert(!(kSum && kMode == kItems), "a unit has one item");
  using R = Ring<kGroup, kZero>;
  constexpr int kEach = R::kEach;
  griddep_begin();
  p.x = after_begin(p.x), p.codes = after_begin(p.codes), p.scale = after_begin(p.scale);
  p.zero = after_begin(p.zero), p.chosen = after_begin(p.chosen), p.weights = after_begin(p.weights);
  p.ready = after_begin(p.ready), p.roots = after_begin(p.roots);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Table table;
  __shared__ float part[kWarps][16][kCols + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slots = p.tokens * p.topk;

  // ---- kStaged: x asked for first, into the place where it is made ready below
  __nv_bfloat16* const staged = reinterpret_cast<__nv_bfloat16*>(smem + kWarps * R::kBytes);
  // this warp's windows, every 16th of the rows' windows in order: each(row, window, this lane's 8 values)
  auto each_window = [&](auto each) {
    int row = 0, w = warp;
    while (w >= p.windows) w -= p.windows, ++row;
#pragma unroll 1
    while (row < p.x_rows) {
      each(row, w, staged + row * p.x_pitch + w * kWindow + lane * 8);
      for (w += kWarps; w >= p.windows; w -= p.windows) ++row;
    }
  };
  if constexpr (kStaged) {
    const int64_t step = p.x_slot != 0 ? p.x_slot : p.x_token;
    each_window([&](int row, int w, __nv_bfloat16* to) {
      const int c = w * kWindow + lane * 8;
      if (c < p.k) copy16(smem_u32(to), p.x + row * step + c);
    });
    copies_commit();
  }

  // ---- items: slots of the same expert in their order, 8 at a time (kSum: those of 8 tokens; a
  // token's second slot of the same expert has an item of its own).  A head is an item's first slot.
  static_assert(kMaxSlots <= kThreads, "a slot a thread");
  if (tid < slots) {
    const int i = tid;
    const int e = p.chosen != nullptr ? p.chosen[i] : 0;
    table.expert[i] = e >= 0 && e < p.experts ? e : -1;
    table.row[i] = int16_t(p.x_slot != 0 ? i : i / p.topk);
    table.columns[i] = 0;
  }
  for (int i = tid; i < kMaxSlots * kCols / 2; i += kThreads) reinterpret_cast<uint32_t*>(table.slot)[i] = 0xFFFFFFFFu;
  uint32_t* tops = reinterpret_cast<uint32_t*>(&part[0][0][0]);  // of the windows of x
  if constexpr (kStaged) {
    copies_wait<0>();
    each_window([&](int row, int w, __nv_bfloat16* at) {
      const uint4 v = w * kWindow + lane * 8 < p.k ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
      const uint32_t top = __reduce_max_sync(0xffffffffu, largest(v));
      if (lane == 0) tops[row * p.windows + w] = top;
    });
  }
  __syncthreads();
  if constexpr (kStaged)
    for (int row = warp; row < p.x_rows; row += kWarps) {
      const int power = power_of(tops + row * p.windows, p.windows);
      if (lane == 0) table.power[row] = int16_t(power);
    }
  // this thread's slot: its expert, its item's head and its column there
  const int columns_of_item = kMode == kItems ? p.item_columns : kCols;
  int mine = -1, head = -1, column = 0;
  if (tid < slots) mine = table.expert[tid];
  if (mine >= 0) {
    head = tid;
    if constexpr (kSum) {
      const int t = tid / p.topk, t0 = t / kCols * kCols;
      column = t - t0;
      int twin = 0;  // earlier slots of the token with this expert
      for (int j = t * p.topk; j < tid; ++j) twin += table.expert[j] == mine;
      // the first token of the eight with so many of them
      for (int u = t0; u < t; ++u) {
        int seen = 0, at = -1;
        for (int j = u * p.topk; j < (u + 1) * p.topk; ++j)
          if (table.expert[j] == mine && seen++ == twin) at = j;
        if (at >= 0) {
          head = at;
          break;
        }
      }
    } else {
      int at = tid;
      for (int j = 0; j < tid; ++j)
        if (table.expert[j] == mine) {
          if (column == 0) at = j;
          column = column + 1 == columns_of_item ? 0 : column + 1;
        }
      head = column == 0 ? tid : at;
    }
  }
  // heads numbered in the order of their slots
  const bool is_head = mine >= 0 && head == tid;
  const uint32_t ballot = __ballot_sync(0xffffffffu, is_head);
  if (lane == 0) table.warp_heads[warp] = __popc(ballot);
  __syncthreads();
  int items = 0, number = __popc(ballot & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) number += table.warp_heads[w];
    items += table.warp_heads[w];
  }
  if (tid < slots) {
    if (kSum && tid % (kCols * p.topk) == 0) table.first[tid / (kCols * p.topk)] = int16_t(number);
    if (is_head) table.number[tid] = int16_t(number), table.head[number] = int16_t(tid), table.item[number] = mine;
  }
  __syncthreads();
  if (mine >= 0) {
    table.slot[table.number[head]][column] = int16_t(tid);
    if constexpr (!kSum) atomicAdd(&table.columns[table.number[head]], 1);
  }
  const int chunks = (p.tokens + kCols - 1) / kCols;
  if (kSum && tid == 0) table.first[chunks] = int16_t(items);
  __syncthreads();

  auto put = [&](int64_t row, int64_t c, float v) {
    if (p.out_f32 != 0)
      static_cast<float*>(p.out)[row * p.out_n + c] = v;
    else
      static_cast<__nv_bfloat16*>(p.out)[row * p.out_n + c] = __float2bfloat16_rn(v);
  };
  if constexpr (!kSum) {  // rows of slots without an expert
    uint32_t none = __ballot_sync(0xffffffffu, tid < slots && mine < 0);
    while (none != 0) {
      const int i = warp * 32 + __ffs(none) - 1;
      none &= none - 1;
      for (int64_t c = int64_t(blockIdx.x) * 32 + lane; c < p.out_n; c += int64_t(gridDim.x) * 32) put(i, c, 0.f);
    }
  }

  // ---- the warp's part of its team's units, in order: pairs of an item and a span
  // warps to a tile: so many that the last team is done first, a unit's start and end counted as a span.
  // Lanes 0 to 4 each look at one power of two.
  const int groups = kSum ? chunks : items;
  int lg = 0;
  {
    const int at = min(lane, 4);
    const unsigned spans = unsigned(p.spans) * (kSum ? (unsigned(items) + chunks - 1) / chunks : 1u);
    const unsigned units = unsigned(groups) * unsigned(min(p.tiles, 1 << 20)), teams = gridDim.x * unsigned(kWarps >> at);
    // (kItems: a CTA's range ends within an item, and in it)
    const unsigned rounds = (units + teams - 1) / teams + (kMode == kItems ? 1 : 0);
    const unsigned each = (spans + (1u << at) - 1) >> at;
    const unsigned total = unsigned(fminf(float(rounds) * float(each + 1), 2.5e8f));
    const unsigned cost = __reduce_min_sync(0xffffffffu, total * 8 + at);
    lg = int(cost % 8);
  }
  const int size = 1 << lg;    // warps of a team
  const int member = warp & (size - 1), team = warp >> lg;
  // teams of all CTAs; a CTA's are far apart, so that the last round is spread over all of them, or next
  // to one another, so that they read the same rows of x through the SM's cache
  const int cta_teams = kWarps >> lg, teams = int(gridDim.x) * cta_teams;
  Unit ahead{0, 0}, here{0, 0};
  int dgroup = 0, dtile = 0;            // between a team's units
  int last_group = 0, last_tiles = 0;   // kItems: the CTA's last group, and how many of its tiles it takes
  if constexpr (kMode == kItems) {  // a range of units for each CTA, its teams side by side within each item
    const int64_t units = int64_t(groups) * p.tiles;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    here.group = int(u0 / p.tiles), here.tile = int(u0 - int64_t(here.group) * p.tiles) + team;
    last_group = int(u1 / p.tiles), last_tiles = int(u1 - int64_t(last_group) * p.tiles);
  } else {
    const int start = kStaged ? int(blockIdx.x) + team * int(gridDim.x) : int(blockIdx.x) * cta_teams + team;
    dgroup = teams / p.tiles, dtile = teams - dgroup * p.tiles;
    here.group = start / p.tiles, here.tile = start - here.group * p.tiles;
  }
  auto tiles_end = [&](int group) { return kMode == kItems && group >= last_group ? last_tiles : p.tiles; };
  auto in_range = [&](const Unit& u) {
    return kMode == kItems ? u.group < last_group || (u.group == last_group && u.tile < last_tiles) : u.group < groups;
  };
  // the team's next unit (kItems: from a place past its tiles, too)
  auto settle = [&](Unit& u) {
    if constexpr (kMode == kItems)
      while (u.group <= last_group && u.tile >= tiles_end(u.group)) u.tile = team, ++u.group;
  };
  auto advance = [&](Unit& u) {
    if constexpr (kMode == kItems) {
      u.tile += cta_teams;
      settle(u);
    } else {
      u.advance(dgroup, dtile, p.tiles);
    }
  };
  const int first_group = here.group;
  settle(here);
  ahead = here;
  uint8_t* const ring = smem + warp * R::kBytes;
  const int lane_row = lane >> 4, lane_chunk = lane & 15;
  // where this lane's pieces of the next span go
  const uint32_t fill_codes = smem_u32(ring) + lane_row * kPitch + lane_chunk * 16;
  const uint32_t fill_lane = smem_u32(ring) + lane * 16;
  uint32_t fill = 0;
  // the pairs of a unit that are this warp's: [begin, end) of its items' spans
  const int begin_one = int((int64_t(p.spans) * member) >> lg), end_one = int((int64_t(p.spans) * (member + 1)) >> lg);
  auto part_of = [&](const Unit& u, int& first, int& begin, int& end) {
    if constexpr (kSum) {
      first = table.first[u.group];
      const int64_t pairs = int64_t(table.first[u.group + 1] - first) * p.spans;
      begin = int((pairs * member) >> lg), end = int((pairs * (member + 1)) >> lg);
    } else {
      first = u.group, begin = begin_one, end = end_one;
    }
  };

  // what is fetched ahead: its pair, and where this lane's pieces are: every other row of codes from
  // lane_row on, and a piece of 8 rows' scales of one of the span's two windows
  constexpr int kPieces = 8 * kEach * 2 / 16, kZeroPieces = kZero ? 8 * kEach / 16 : 1;
  const int whole = p.k / kSpan;
  const int64_t pitch = p.k / 2, scale_step = int64_t(p.n) * kEach * 2;
  int pair = 0, pair_end = 0, item = 0, span = 0;
  bool second = false;  // the tile has its second 8 rows
  const uint8_t *code0 = nullptr, *code1 = nullptr, *scale = nullptr, *zero = nullptr;
  auto aim = [&] {
    const int64_t e = table.item[item];
    const int row0 = kGated ? ahead.tile * 8 : ahead.tile * 16;
    second = kGated || row0 + 8 < p.n;
    const int row1 = !second ? row0 : kGated ? p.n / 2 + row0 : row0 + 8;
    const uint8_t* at = p.codes + (e * p.n + lane_row) * pitch + int64_t(span) * (kSpan / 2) + lane_chunk * 16;
    code0 = at + row0 * pitch, code1 = at + row1 * pitch;
    const int64_t in_window = (e * p.windows + 2 * int64_t(span)) * p.n;
    const int64_t of_scales = in_window + int64_t(lane / (2 * kPieces)) * p.n + (lane / kPieces % 2 ? row1 : row0);
    scale = p.scale + of_scales * (kEach * 2) + lane % kPieces * 16;
    if constexpr (kZero) {
      const int64_t of_zeros = in_window + int64_t(lane / (2 * kZeroPieces)) * p.n + (lane / kZeroPieces % 2 ? row1 : row0);
      zero = p.zero + of_zeros * kEach + lane % kZeroPieces * 16;
    }
  };
  auto enter = [&] {
    while (in_range(ahead)) {
      int first;
      part_of(ahead, first, pair, pair_end);
      if (pair < pair_end) {
        const int skip = kSum ? pair / p.spans : 0;
        item = first + skip, span = pair - skip * p.spans;
        aim();
        return;
      }
      advance(ahead);
    }
  };
  auto fetch = [&] {  // and on to the next
    if (in_range(ahead)) {
      const uint32_t to = fill_codes + fill, to_lane = fill_lane + fill;
      if (second && span < whole) {
        const uint8_t *c0 = code0, *c1 = code1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          copy16(to + 2 * i * kPitch, c0);
          copy16(to + (8 + 2 * i) * kPitch, c1);
          c0 += 2 * pitch, c1 += 2 * pitch;
        }
        if (lane < 4 * kPieces) copy16(to_lane + R::kScaleAt, scale);
        if constexpr (kZero)
          if (lane < 4 * kZeroPieces) copy16(to_lane + R::kZeroAt, zero);
      } else {  // zeros for what is past k or n, with an address inside
        const bool in = span * kSpan + lane_chunk * 32 < p.k, two = 2 * span + 1 < p.windows;
        const int64_t back = in ? 0 : lane_chunk * -16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          copy16(to + 2 * i * kPitch, code0 + 2 * i * pitch + back, in);
          copy16(to + (8 + 2 * i) * kPitch, code1 + 2 * i * pitch + back, in && second);
        }
        if (lane < 4 * kPieces) {
          const bool there = (two || lane < 2 * kPieces) && (second || lane / kPieces % 2 == 0);
          copy16(to_lane + R::kScaleAt, there ? scale : p.scale, there);
        }
        if constexpr (kZero) {
          if (lane < 4 * kZeroPieces) {
            const bool there = (two || lane < 2 * kZeroPieces) && (second || lane / kZeroPieces % 2 == 0);
            copy16(to_lane + R::kZeroAt, there ? zero : p.zero, there);
          }
        }
      }
      fill = R::kStage - fill;
      if (++pair == pair_end) {
        advance(ahead);
        enter();
      } else if (++span == p.spans) {
        span = 0, ++item;
        aim();
      } else {
        code0 += kSpan / 2, code1 += kSpan / 2, scale += 2 * scale_step;
        if constexpr (kZero) zero += scale_step;
      }
    }
    copies_commit();
  };
  enter();
  fetch();

  // rows of x made ready: in shared memory, or by the kernel ahead
  const __nv_bfloat16* ready = p.ready;
  const float* roots = p.roots;
  if constexpr (kStaged) {
    auto* to_roots = reinterpret_cast<float*>(staged + p.x_rows * p.x_pitch);
    ready = staged, roots = to_roots;
    each_window([&](int row, int w, __nv_bfloat16* at) {
      const uint4 v = w * kWindow + lane * 8 < p.k ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
      make_ready(v, p.k, w, table.power[row], staged + row * p.x_pitch);
    });
    if (tid < p.x_rows) to_roots[tid] = root_of(table.power[tid]);
    __syncthreads();
  }

  const int g = lane >> 2, t4 = lane & 3;
  auto team_sync = [&] {
    if (lg == 0)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(32 << lg) : "memory");
  };
  int last = -1;
  const uint8_t* const words = ring + g * kPitch + t4 * 4;  // this lane's words of a stage
  const int scale_off = R::kScaleAt + g * kEach * 2 - g * kPitch - t4 * 4;
  const int zero_off = R::kZeroAt + g * kEach - g * kPitch - t4 * 4;
  int stage = 0;
  // two's complement + 8 is the top bit flipped
  const uint32_t mask_low = in_register(0x000F000Fu), mask_high = in_register(0x00F000F0u);
  const uint32_t flip_low = in_register(0x00080008u), flip_high = in_register(0x00800080u);
  const uint32_t up_low = in_register(0x4B004B00u), up_high = in_register(0x49004900u);  // 2^23, 2^19
  const __nv_bfloat16* xp = nullptr;  // column g of the last item, from this lane's k on
  float w0 = 0.f, w1 = 0.f, root0 = 0.f, root1 = 0.f;
  bool has0 = false, has1 = false;
  auto work = [&] {  // on the unit here
    int first, at, end;
    part_of(here, first, at, end);
    int now = first + (kSum ? at / p.spans : 0), w = kSum ? at - (now - first) * p.spans : at;
    float res[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (; at < end; ++at) {
      if (now != last) {
        last = now;
        // a column without a slot takes the head's x: nothing of it is used
        const int s = table.slot[now][g], s0 = table.slot[now][2 * t4], s1 = table.slot[now][2 * t4 + 1];
        has0 = s0 >= 0, has1 = s1 >= 0;
        const int head = table.row[table.head[now]];
        // column g's row of x: of the item's, or of all
        const int r = kMode == kItems ? (s < 0 ? 0 : g) : s < 0 ? head : table.row[s];
        xp = ready + int64_t(r) * (kMode == kItems ? p.item_pitch : p.x_pitch) + t4 * 8;
        if constexpr (kSum) {
          w0 = has0 ? p.weights[s0] : 0.f, w1 = has1 ? p.weights[s1] : 0.f;
          root0 = roots[has0 ? table.row[s0] : head], root1 = roots[has1 ? table.row[s1] : head];
        }
      }
      const int k0 = w * kSpan;
      const __nv_bfloat16* xk = xp + k0;
      // x of the next two chunks is read ahead of its use, where it may come from the L2
      constexpr int kQuad = 128 / kGroup;  // groups of four chunks
      uint4 b[2][2];
      auto read_x = [&](int pair) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          b[pair % 2][i] = load<kShared>(reinterpret_cast<const uint4*>(xk + (pair * 2 + i) * 32));
      };
      const bool full = k0 + kSpan <= p.k;
      if (!kShared && full) read_x(0);
      copies_wait<0>();
      __syncwarp();
      fetch();
      const uint8_t *codes = words + stage, *scales = codes + scale_off, *zeros = codes + zero_off;
      stage = R::kStage - stage;
      constexpr uint32_t kEight = 0x8A008A00u;  // -2^-110 times 8
      auto off_of = [&](uint32_t z) { return fma2(z, 0xCB00CB00u, 0); };
      // one group, its chunks' x given by `x_of`
      // (z0, z1: -2^-110 times the zero points of rows g and g + 8, twice each)
      auto group = [&](int q, float s0, float s1, uint32_t z0, uint32_t z1, auto x_of) {
        auto low = [&](uint32_t v, uint32_t z) {
          return fma2(kZero ? v & mask_low : masked(v, mask_low, flip_low), up_low, z);
        };
        auto high = [&](uint32_t v, uint32_t z) {
          return fma2(kZero ? v & mask_high : masked(v, mask_high, flip_high), up_high, z);
        };
        float c[4];
#pragma unroll
        for (int j = 0; j < kGroup / 32; ++j) {
          const int chunk = q * (kGroup / 32) + j;
          const uint4 v = x_of(chunk);
          const uint32_t wa = *reinterpret_cast<const uint32_t*>(codes + chunk * 16), va = wa >> 8;
          const uint32_t wb = *reinterpret_cast<const uint32_t*>(codes + 8 * kPitch + chunk * 16), vb = wb >> 8;
          mma(c, low(wa, z0), low(wb, z1), high(wa, z0), high(wb, z1), v.x, v.y, j == 0);
          mma(c, low(va, z0), low(vb, z1), high(va, z0), high(vb, z1), v.z, v.w, false);
        }
        acc[0] = fmaf(s0, c[0], acc[0]), acc[1] = fmaf(s0, c[1], acc[1]);
        acc[2] = fmaf(s1, c[2], acc[2]), acc[3] = fmaf(s1, c[3], acc[3]);
      };
      if (full) {
        using Scales = std::conditional_t<kEach == 2, uint32_t, std::conditional_t<kEach == 4, uint2, uint4>>;
        Scales sa, sb;
        using Zeros = std::conditional_t<kEach == 2, uint16_t, std::conditional_t<kEach == 4, uint32_t, uint2>>;
        uint32_t za[2] = {0, 0}, zb[2] = {0, 0};
        auto zeros_of = [](uint32_t (&z)[2], const Zeros& v) {
          if constexpr (kEach == 8)
            z[0] = v.x, z[1] = v.y;
          else
            z[0] = v;
        };
#pragma unroll
        for (int quad = 0; quad < 4; ++quad) {
          if (quad % 2 == 0) {
            sa = reinterpret_cast<const Scales*>(scales)[8 * quad];
            sb = reinterpret_cast<const Scales*>(scales)[8 * quad + 8];
            if constexpr (kZero) {
              zeros_of(za, reinterpret_cast<const Zeros*>(zeros)[8 * quad]);
              zeros_of(zb, reinterpret_cast<const Zeros*>(zeros)[8 * quad + 8]);
            }
          }
#pragma unroll
          for (int i = 0; i < kQuad; ++i) {
            const int at = quad % 2 * kQuad + i;  // in the window
            const uint32_t pa = reinterpret_cast<const uint32_t*>(&sa)[at / 2];
            const uint32_t pb = reinterpret_cast<const uint32_t*>(&sb)[at / 2];
            group(quad * kQuad + i, __uint_as_float(at % 2 ? pa & 0xFFFF0000u : pa << 16),
                  __uint_as_float(at % 2 ? pb & 0xFFFF0000u : pb << 16),
                  kZero ? off_of(__byte_perm(za[at / 4], 0, 0x4040u + at % 4 * 0x0101u)) : kEight,
                  kZero ? off_of(__byte_perm(zb[at / 4], 0, 0x4040u + at % 4 * 0x0101u)) : kEight, [&](int chunk) {
                    if constexpr (kShared) return load<true>(reinterpret_cast<const uint4*>(xk + chunk * 32));
                    if (chunk % 2 == 0 && chunk < 14) read_x(chunk / 2 + 1);
                    return b[chunk / 2 % 2][chunk % 2];
                  });
          }
        }
      } else {
        const __nv_bfloat16* one = reinterpret_cast<const __nv_bfloat16*>(scales);
        const int left = (p.k - k0) / kGroup;
#pragma unroll 1
        for (int q = 0; q < left; ++q) {
          const int sq = q / kEach * (16 * kEach) + q % kEach;
          uint32_t z0 = kEight, z1 = kEight;
          if constexpr (kZero) z0 = off_of(zeros[sq] * 0x00010001u), z1 = off_of(zeros[8 * kEach + sq] * 0x00010001u);
          group(q, __bfloat162float(one[sq]), __bfloat162float(one[8 * kEach + sq]), z0, z1,
                [&](int chunk) { return load<kShared>(reinterpret_cast<const uint4*>(xk + chunk * 32)); });
        }
      }
      if (!kSum) {
        ++w;
      } else if (++w == p.spans || at + 1 == end) {
        if (has0) res[0] += w0 * (acc[0] * root0 * root0), res[2] += w0 * (acc[2] * root0 * root0);
        if (has1) res[1] += w1 * (acc[1] * root1 * root1), res[3] += w1 * (acc[3] * root1 * root1);
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
        if (w == p.spans) w = 0, ++now;
      }
    }
    const float* mine4 = kSum ? res : acc;
    team_sync();  // the last unit's sums have been read
    part[warp][g][2 * t4] = mine4[0], part[warp][g][2 * t4 + 1] = mine4[1];
    part[warp][g + 8][2 * t4] = mine4[2], part[warp][g + 8][2 * t4 + 1] = mine4[3];
    team_sync();
    // sums over the team's warps, and out
    constexpr int kRows = kGated ? 8 : 16;
    const int columns = kSum ? p.tokens - here.group * kCols : table.columns[here.group];
    const float* sum = &part[team << lg][0][0];
    for (int i = member * 32 + lane; i < kRows * min(columns, kCols); i += 32 << lg) {
      const int row = i % kRows, col = i / kRows;
      const int64_t c = int64_t(here.tile) * kRows + row;
      if (c >= p.out_n) continue;
      const float* from = sum + row * (kCols + 1) + col;
      float v = 0.f, u = 0.f;
      for (int m = 0; m < size; ++m) {
        v += from[m * 16 * (kCols + 1)];
        if constexpr (kGated) u += from[(m * 16 + 8) * (kCols + 1)];
      }
      if constexpr (kSum) {
        put(here.group * kCols + col, c, v);
      } else {
        const int to = table.slot[here.group][col];
        const float root = roots[table.row[to]];
        v = v * root * root;
        if constexpr (kGated) {
          u = u * root * root;
          v = (p.act == GMM_ACT_SILU ? act_value<GMM_ACT_SILU, false>(v) : act_value<GMM_ACT_GELU, false>(v)) * u;
        }
        put(to, c, v);
      }
    }
  };
  if constexpr (kMode == kItems) {
    auto* rows = reinterpret_cast<__nv_bfloat16*>(smem + kWarps * R::kBytes);
    const int eights = p.k / 8;
    ready = rows;
    for (int group = first_group; group <= last_group && (group < last_group || last_tiles > 0); ++group) {
      __syncthreads();  // the last item's x has been read
      const int columns = table.columns[group];
      for (int c = 0; c < columns; ++c) {
        const int64_t row = table.row[table.slot[group][c]];
        for (int i = tid; i < eights; i += kThreads)
          copy16(smem_u32(rows + c * p.item_pitch + i * 8), p.ready + row * p.x_pitch + i * 8);
      }
      copies_commit();
      copies_wait<0>();
      __syncthreads();
      last = -1;
      for (; here.group == group && in_range(here); advance(here)) work();
    }
  } else {
    for (; in_range(here); advance(here)) work();
  }
  copies_wait<0>();
}

// Rows of x made ready where a CTA's shared memory does not hold them: a CTA a row.
__global__ void __launch_bounds__(kThreads) make_ready_kernel(Params p) {
  griddep_begin();
  p.x = after_begin(p.x);
  __shared__ uint32_t tops[kWarps];
  const int row = blockIdx.x, warp = threadIdx.x >> 5;
  const __nv_bfloat16* x = p.x + row * (p.x_slot != 0 ? p.x_slot : p.x_token);
  uint32_t top = 0;
#pragma unroll 4
  for (int w = warp; w < p.windows; w += kWarps) top = max(top, largest(window_of(x, p.k, w)));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) tops[warp] = top;
  __syncthreads();
  const int power = power_of(tops, kWarps);
#pragma unroll 4
  for (int w = warp; w < p.windows; w += kWarps)
    make_ready(window_of(x, p.k, w), p.k, w, power, p.ready + int64_t(row) * p.x_pitch);
  if (threadIdx.x == 0) p.roots[row] = root_of(power);
}

constexpr size_t kMaxShared = 227 * 1024 - 256 - sizeof(Table) - sizeof(float) * kWarps * 16 * (kCols + 1);

// Bytes of `rows` rows of x made ready, `pitch` elements apart: the values, the roots.
int64_t ready_bytes(int64_t rows, int64_t pitch) { return rows * (pitch * 2 + 4); }
// In shared memory rows are half a line of banks apart.
int64_t staged_pitch(int64_t k) { return k % 64 == 0 ? k + 32 : k; }
// Rows that fit the shared memory.
int64_t staged_rows(int64_t k, int group, bool zero) {
  const int64_t each = kWindow / group, ring = int64_t(kWarps) * 2 * (16 * kPitch + 2 * 16 * each * (zero ? 3 : 2));
  return (int64_t(kMaxShared) - ring) / ready_bytes(1, staged_pitch(k));
}
int64_t launch_tokens(int64_t topk) { return kMaxSlots / topk / kCols * kCols; }

template <int kGroup, bool kZero, bool kGated, bool kSum, Mode kMode>
cudaError_t launch(const Params& p, int sms, cudaStream_t stream) {
  using R = Ring<kGroup, kZero>;
  const int64_t rows = kMode == kAll ? p.x_rows : kMode == kItems ? p.item_columns : 0;
  const size_t smem = size_t(kWarps) * R::kBytes + size_t(ready_bytes(rows, staged_pitch(p.k)));
  auto kern = matvec_kernel<kGroup, kZero, kGated, kSum, kMode>;
  // for every launch: the attribute is the current device's, and one size for all calls
  if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxShared))) return e;
  if constexpr (kMode != kAll)
    if (cudaError_t e = launch_dependent(make_ready_kernel, unsigned(p.x_rows), kThreads, 0, stream, 1, p)) return e;
  return launch_dependent(kern, unsigned(sms), kThreads, smem, stream, 1, p);
}

template <int kGroup, bool kZero, bool kGated, bool kSum>
cudaError_t by_mode(Params p, int sms, cudaStream_t stream) {
  const int64_t fit = staged_rows(p.k, kGroup, kZero);
  if (p.x_rows <= fit) return launch<kGroup, kZero, kGated, kSum, kAll>(p, sms, stream);
  if constexpr (!kSum) {
    // Copying an item's x pays where a CTA then has at least some 50 spans of weights for its warps (experts
    // counted at most once): 16 tokens, 2 of 8 experts of 4096 x 4096 (108 spans) take 22.3 us and through the
    // caches 24.9, 32 of 4 of 16 of 1024 x 1024 (13; it fits as a whole, but put through both) 14.1 and 11.3.
    // Fewer columns than half of an item's would read the weights more than twice as often.
    const int64_t items = p.experts < p.tokens * p.topk ? p.experts : p.tokens * p.topk;
    p.item_columns = int32_t(fit < kCols ? fit : kCols), p.item_pitch = int32_t(staged_pitch(p.k));
    if (p.item_columns >= kCols / 2 && items * p.tiles * p.spans >= 50 * int64_t(sms))
      return launch<kGroup, kZero, kGated, kSum, kItems>(p, sms, stream);
  }
  return launch<kGroup, kZero, kGated, kSum, kCaches>(p, sms, stream);
}

template <int kGroup, bool kZero>
cudaError_t by_form(const Params& p, int sms, cudaStream_t stream) {
  if (p.weights != nullptr) return by_mode<kGroup, kZero, false, true>(p, sms, stream);
  return p.act != GMM_ACT_NONE ? by_mode<kGroup, kZero, true, false>(p, sms, stream)
                               : by_mode<kGroup, kZero, false, false>(p, sms, stream);
}

cudaError_t matvec(const Params& p, int group, int sms, cudaStream_t stream) {
  const bool zero = p.zero != nullptr;
  switch (group) {
    case 32: return zero ? by_form<32, true>(p, sms, stream) : by_form<32, false>(p, sms, stream);
    case 64: return zero ? by_form<64, true>(p, sms, stream) : by_form<64, false>(p, sms, stream);
    default: return zero ? by_form<128, true>(p, sms, stream) : by_form<128, false>(p, sms, stream);
  }
}

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

}  // namespace
}  // namespace gmmk

extern "C" size_t gmm_matvec_scratch_bytes(int64_t tokens, int64_t k, int32_t group, int has_zero, int32_t topk,
                                           int x_per_slot) {
  using namespace gmmk;
  if (tokens <= 0 || tokens > kMaxSize || k < 1 || k > kMaxSize || (group != 32 && group != 64 && group != 128) ||
      topk < 1 || topk > GMM_MAX_TOPK)
    return 0;
  const int64_t most = launch_tokens(topk), count = tokens < most ? tokens : most;
  const int64_t rows = x_per_slot != 0 ? count * topk : count;
  // a last launch of fewer tokens may not need what the others do
  // the size it has had: four more bytes for each group of a row than are used
  return rows <= staged_rows(k, group, has_zero != 0) ? 0 : size_t(ready_bytes(rows, k) + rows * ((k / group + 3) / 4 * 16));
}

extern "C" int gmm_matvec_int4(const void* x, int64_t tokens, int64_t k, int64_t x_ld, int x_per_slot, const void* codes,
                               const void* scale, const void* zero, int32_t group, int32_t num_experts, int64_t n,
                               const int32_t* experts, int32_t topk, const float* weights, int act, void* out,
                               int out_dtype, void* scratch, size_t scratch_bytes, void* stream) {
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
  if (misaligned(scratch, 16)) return GMM_ERR_ALIGN;
  const size_t needed = gmm_matvec_scratch_bytes(tokens, k, group, zero != nullptr, topk, x_per_slot);
  if (scratch_bytes < needed || (needed > 0 && scratch == nullptr)) return GMM_ERR_WORKSPACE;
  int sms = 0;
  if (int st = require_device(&sms)) return st;
  const int64_t out_n = act != GMM_ACT_NONE ? n / 2 : n;
  const int64_t most = launch_tokens(topk);
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t count = tokens - t0 < most ? tokens - t0 : most;
    Params p{};
    p.x_token = x_per_slot != 0 ? k * topk : x_ld, p.x_slot = x_per_slot != 0 ? k : 0;
    p.x = static_cast<const __nv_bfloat16*>(x) + t0 * p.x_token;
    p.codes = static_cast<const uint8_t*>(codes), p.scale = static_cast<const uint8_t*>(scale);
    p.zero = static_cast<const uint8_t*>(zero);
    p.experts = num_experts, p.n = int32_t(n), p.k = int32_t(k), p.windows = int32_t((k + kWindow - 1) / kWindow);
    p.spans = int32_t((k + kSpan - 1) / kSpan);
    p.tiles = int32_t((n + 15) / 16);
    p.chosen = experts == nullptr ? nullptr : experts + t0 * topk;
    p.tokens = int32_t(count), p.topk = topk;
    p.weights = weights == nullptr ? nullptr : weights + t0 * topk;
    p.act = act, p.out_n = int32_t(out_n), p.out_f32 = out_dtype == GMM_DTYPE_F32;
    p.x_rows = int32_t(x_per_slot != 0 ? count * topk : count);
    const bool staged = p.x_rows <= staged_rows(k, group, zero != nullptr);
    p.x_pitch = int32_t(staged ? staged_pitch(k) : k);
    if (!staged) {
      p.ready = static_cast<__nv_bfloat16*>(scratch);
      p.roots = reinterpret_cast<float*>(p.ready + int64_t(p.x_rows) * k);
    }
    const int64_t first = t0 * (weights != nullptr ? 1 : topk) * out_n;
    p.out = static_cast<char*>(out) + first * (out_dtype == GMM_DTYPE_F32 ? 4 : 2);
    const cudaError_t e = matvec(p, group, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return record_cuda_error(e);
  }
  return GMM_OK;
}
