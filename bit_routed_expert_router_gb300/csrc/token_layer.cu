// A routed layer and its shared expert for up to 32 tokens, in two kernels:
//
//   up     a[i] = gate GELU(g) u,  [g, u] = Wgu[e] x[t]     for the tokens of each picked expert, in 16 bits
//   down   y[t] = sum_e Wd[e] a[e, t]                       over the experts that t names, and the shared one
//
// a is rounded because it is an operand of 16-bit products and two bytes of the
// workspace.  With 16-bit weights it has their type: the output's error is 1.4 roundings
// of it instead of one.  With e4m3 weights, which are exact in either type, it is fp16
// whatever the call's: one rounding of bf16, and they are widened to it in a third of
// the instructions.  (As two digits, a high and a low operand with an exponent for each
// eight values in the same two bytes, which is 2^-13: one token 27.4 -> 30.4 us.)  What
// leaves fp16's range takes another form in the same place, see Packed.
//
// The weights of the picked experts are read once and nothing else is of any
// size, so both kernels stream them.  A warp works by itself: one of its lanes
// loads chunks of 16 weight rows by TMA into the warp's own stages, and the warp
// multiplies them as m16n8k16 fragments, weights on the M side.  No barrier but a
// stage's own is waited for on the way (with eight warps that shared the stages and
// a ninth that loaded, one token took 47 us instead of 30).  The
// token rows come from L2 straight into fragments, before the chunk's weights are
// waited for (staged beside the weights they took their room: 7 tokens 144 us).
// A lane reads 16 bytes of a row at a time: the order of k within a step is the
// same in both operands, which is all that a product needs.  The rows of a fragment
// are dealt to the lanes so that eight lanes that read at once find the two rows'
// halves of the 128-byte swizzle in different banks.  e4m3 weights become 16-bit
// ones in registers (exact); the sums of each block of 128 are scaled by themselves.
//
// The columns are up to eight tokens of an expert (a slot: an expert with more
// has several, whose weights come from L2 again), so that weights that are not
// finite reach the tokens that name their expert only.
//
// up: a unit is 8 features of a slot: their 8 gate and 8 up rows are the 16 rows,
// so that a lane ends with both factors of its values.
// down: a unit is 16 outputs over all slots, its chunks dealt out to the warps of a
// cluster's CTAs.  Each adds its slots' sums to its own copy of the tokens'
// outputs; the copies are added in order, through distributed shared memory.  The
// kernel starts on an SM as the first one leaves it, and fills its stages with
// weights while others still run.
//
// 128 experts of 2816 x 704, 8 of them a token, and a shared one of 2816 x 2816: 7
// tokens 85 us in a graph, HBM; one token 27.4 us (143 MB, 5.2 TB/s), in 8 bits 20.4
// (71 MB, 3.5 TB/s).  What nothing hides there: 2.3 us from the start to the first
// weights, 3 us from one kernel's last sums to the other's first weights (with
// stages of 64 KB, which fit beside the first kernel's, and all of the SM's shared
// memory set as such the second starts early, but takes HBM from the first: 28.5 us
// at 27.9), 1 us of tails; in 8 bits the first kernel's widening.
#include <algorithm>
#include <type_traits>

#include "allow_smem.h"
#include "gelu16.cuh"
#include "grouped.h"
#include "ops8.h"
#include "tc16.cuh"
#include "tensor_map.h"
#include "waits.cuh"

namespace moe {

namespace {

using tc16::cluster_rank;
using tc16::cluster_sync;
using tc16::elect_one;

constexpr int kTeams = 8, kWarpsDown = 8;          // units that a CTA of the first kernel has at hand; warps of the second's
// Warps of a team, which take a unit's chunks in turn where it has several.  Widening e4m3 is a chain of four instructions: with
// one warp a unit, two a scheduler, it held the weights up (8 bits, one token, 23.5 -> 21.9 us; with 88 registers a thread instead of 128 25.5).
constexpr int team_of(bool w8) { return w8 ? 2 : 1; }
constexpr int kTeamStages = 2, kStagesDown = 1;    // chunks on their way: of a team, of a warp
constexpr int kCol = 128, kColBytes = 16 * kCol;  // bytes of a weight row that one load takes; of its 16 rows
// Loads of a chunk: neighbours in their rows, which the memory likes (chunks of 256 bytes of a row 34 us for one token, 104 for
// seven, when those of 512 took 29.8 and 87.9; in the second kernel 768 bytes instead of 512 27.6 -> 27.1 and 83.5 -> 83.1).
constexpr int kColsUp = 4, kColsDown = 6;
// The type of a: fp16, or bf16.
constexpr bool half_a(bool bf16, bool w8) { return w8 || !bf16; }
// Of these, loads whose token values a lane holds at a time (registers: two CTAs of the second kernel an SM).
constexpr int kTokensUp = kColsUp;
constexpr int tokens_down(bool w8) { return w8 ? 3 : kColsDown; }
constexpr int kTokens = 8;                       // of a slot
constexpr int kMostSplit = 8;                    // CTAs that share a unit of the second kernel
constexpr int kMostSmem = 160 * 1024;            // of either kernel: the stages, and the lists of 1024 pairs and experts

struct Slot {
  int expert;      // -1: the shared expert
  uint32_t mask;   // its tokens, kTokens at most
  int base;        // its rows of a (the shared one's: in its own part)
};

// What a launch's CTA keeps behind the stages, and where.
struct Plan {
  int at_sums, at_mask, at_ids, at_gates, at_slots, bytes;
};

__host__ __device__ __forceinline__ int divide_up(int a, int b) { return (a + b - 1) / b; }

template <int kWarps, int kStages>
struct Shared {
  uint64_t full[kWarps][kStages];
  Waits waits;
  int n_routed, n_slots;   // slots of routed experts; and of the shared one
};

// ------------------------------------------------------------------ pieces

template <bool kBf16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 values in the call's type (exact in both).
template <bool kBf16>
__device__ __forceinline__ uint32_t widen8(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  if (!kBf16) return h;
  const __nv_bfloat162 b = __floats2bfloat162_rn(half_lo(h), half_hi(h));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The weight row of a fragment's row g (and 8 + it that of row 8 + g).
__device__ __forceinline__ int row_of(int g) { return g >> 1 | (g & 1) << 2; }

// This lane's share of up to 8 token rows over a chunk: 16 bytes a word.
template <bool kW8, int kCols>
struct TokenWords {
  static constexpr int kWords = kW8 ? 2 : 1;   // of a half of a load
  uint4 v[kCols][2][kWords];

  // row: this lane's token row from the chunk's first value on, of which k are there (a lane without a token of its own takes
  // another's: its column is not used)
  __device__ __forceinline__ void load(const uint16_t* row, int k, int lane) {
    const int at = 8 * kWords * (lane & 3);
    if (k >= (kW8 ? kCol : kCol / 2) * kCols)
      take<true>(row + at, k - at);
    else
      take<false>(row + at, k - at);
  }
  template <bool kWhole>
  __device__ __forceinline__ void take(const uint16_t* row, int k) {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const int at = (kW8 ? kCol : kCol / 2) * i + 32 * kWords * h + 8 * j;
          v[i][h][j] = kWhole || at < k ? __ldcg(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0, 0, 0, 0);
        }
  }
  // what the sums of this lane's column `column` are to be multiplied by
  __device__ __forceinline__ float unit(int) const { return 1.f; }
};

// ------------------------------------------------------------------ a in fp16
//
// Eight features of a token (a unit's, 16 bytes) are fp16 values if the largest is 0 or from 2^-13 on in fp16's range: none is
// off by more than half a step or 2^-12 of the largest.  Others are packed, which the last value's exponent tells (infinity's,
// which no value has): under it, in its fraction, lies e = k + 127 > 0, with 2^k <= |v| < 2^(k+1) for the largest once rounded; the
// others' words hold integers v 2^(12-k), 14 bits, and above each of them two bits of the last one's.  To a product that takes
// it for a value the last one's word is NaN, and so is the product.  (All of one token's packed: 28 -> 44 us, of seven tokens' 85
// -> 143.)
struct Packed {
  static constexpr uint32_t kMark = 0x7C00;
  static constexpr uint32_t kSmall = 0x39000000u, kLarge = 0x477FF000u;   // 2^-13; 65520, which would round to infinity
  static constexpr int kLeast = 27, kMost = 254;   // of e; below 2^-100 values lose bits, then become 0
  static constexpr uint32_t kNotFinite = 255;      // e: the integers 1, -1, 2 are infinity, -infinity, NaN, and 0 what is finite
                                                   // (no sum that it goes into is)
  static __device__ __forceinline__ bool needed(uint32_t top) { return top && top - kSmall >= kLarge - kSmall; }
  // e from the largest magnitude's bits
  static __device__ __forceinline__ uint32_t exponent(uint32_t top) {
    if (top >= 0x7F800000u) return kNotFinite;
    return min(max((top + (1u << 10)) >> 23, static_cast<uint32_t>(kLeast)), static_cast<uint32_t>(kMost));
  }
  static __device__ __forceinline__ int integer(float v, uint32_t e) {
    if (e == kNotFinite) return isnan(v) ? 2 : !isinf(v) ? 0 : v > 0.f ? 1 : -1;
    return min(__float2int_rn(v * __uint_as_float((kMost + 12 - e) << 23)), 8191);
  }
  // the word of feature i from its integer and the last feature's
  static __device__ __forceinline__ uint16_t word(int i, int own, int last, uint32_t e) {
    return static_cast<uint16_t>(i == 7 ? kMark | e : (own & 0x3FFF) | (last >> 2 * i & 3) << 14);
  }
  static __device__ __forceinline__ bool is(const uint4& v) { return (v.w >> 16 & kMark) == kMark; }
  // e of eight words, packed or not (of fp16's smallest values that of 2^-15); 0: zeros, or not finite
  static __device__ __forceinline__ int exponent(const uint4& v) {
    if (is(v)) return (v.w >> 16 & 0x3FF) == kNotFinite ? 0 : v.w >> 16 & 0x3FF;
    const uint32_t m = 0x7FFF7FFF, top = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return top ? 112 + (max(top >> 16, top & 0xFFFF) >> 10) : 0;
  }
  // two of their values each, times a power of two, as fp16
  static __device__ __forceinline__ uint4 scaled(const uint4& v, float by) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[4];
    const auto pair = [&](int i, float lo, float hi) {
      const __half2 two = __floats2half2_rn(lo, hi);
      out[i] = *reinterpret_cast<const uint32_t*>(&two);
    };
    if (!is(v)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) pair(i, half_lo(w[i]) * by, half_hi(w[i]) * by);
    } else {
      const uint32_t e = v.w >> 16 & 0x3FF;
      int m[8];
      uint32_t last = 0;
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        const uint32_t bits = i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFF;
        last |= bits >> 14 << 2 * i;
        m[i] = static_cast<int>(bits << 18) >> 18;
      }
      m[7] = static_cast<int>(last << 18) >> 18;
      if (e != kNotFinite) {
        const float step = __uint_as_float((e - 12) << 23) * by;
#pragma unroll
        for (int i = 0; i < 4; ++i) pair(i, static_cast<float>(m[2 * i]) * step, static_cast<float>(m[2 * i + 1]) * step);
      } else {
        const auto value = [](int m) { return m == 0 ? 0.f : __int_as_float(m == 2 ? 0x7FC00000 : m > 0 ? 0x7F800000 : 0xFF800000); };
#pragma unroll
        for (int i = 0; i < 4; ++i) pair(i, value(m[2 * i]), value(m[2 * i + 1]));
      }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};

// TokenWords of a of which some may be packed: `scale` makes them the values by the power of two that brings the largest of this
// lane's token under 2^15; `units` takes it out of the sums again.  What is 2^-29 of the largest loses bits.
template <bool kW8, int kCols>
struct ScaledWords : TokenWords<kW8, kCols> {
  using Words = TokenWords<kW8, kCols>;
  float units[2];

  __device__ __forceinline__ uint4& word(int i) { return this->v[i / (2 * Words::kWords)][i / Words::kWords % 2][i % Words::kWords]; }
  __device__ __forceinline__ void scale(int lane) {
    int e = Packed::kLeast;
#pragma unroll
    for (int i = 0; i < kCols * 2 * Words::kWords; ++i) e = max(e, Packed::exponent(word(i)));
    e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
    e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
    const float by = __int_as_float((268 - e) << 23);   // 2^(14 - k)
#pragma unroll
    for (int i = 0; i < kCols * 2 * Words::kWords; ++i) word(i) = Packed::scaled(word(i), by);
#pragma unroll
    for (int i = 0; i < 2; ++i) units[i] = __int_as_float((__shfl_sync(0xFFFFFFFFu, e, 8 * (lane & 3) + 4 * i) - 14) << 23);
  }
  __device__ __forceinline__ float unit(int column) const { return units[column]; }
};

// acc += 16 weight rows of staged loads of k values times the token rows.  With e4m3 weights `scale` holds the scales of the
// chunk's blocks of 128 (its loads, these from `block` on): lane i that of rows 0 .. 7, lane 16 + i of rows 8 .. 15.
template <bool kBf16, bool kW8, int kCols, typename Words>
__device__ __forceinline__ void chunk_products(float (&acc)[4], const uint8_t* stage, const Words& x, int k, float scale, int block,
                                               int lane) {
  const int r = row_of(lane >> 2), t = lane & 3;
  const uint8_t* row = stage + r * kCol;
  float part[2][4] = {};
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    if ((kW8 ? kCol : kCol / 2) * i >= k) break;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* from = row + i * kColBytes + (((4 * h + t) ^ r) << 4);   // zeros past the row's end
      const uint4 w0 = *reinterpret_cast<const uint4*>(from), w1 = *reinterpret_cast<const uint4*>(from + 8 * kCol);
      const uint4 b0 = x.v[i][h][0];
      if (kW8) {
        const uint4 b1 = x.v[i][h][Words::kWords - 1];
        const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
        const uint32_t b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma16<kBf16>(part[h], widen8<kBf16>(lo[q]), widen8<kBf16>(hi[q]), widen8<kBf16>(lo[q] >> 16), widen8<kBf16>(hi[q] >> 16),
                       b[2 * q], b[2 * q + 1]);
      } else {
        mma16<kBf16>(part[h], w0.x, w1.x, w0.y, w1.y, b0.x, b0.y);
        mma16<kBf16>(part[h], w0.z, w1.z, w0.w, w1.w, b0.z, b0.w);
      }
    }
    if (kW8) {
      const float lo = __shfl_sync(0xFFFFFFFFu, scale, block + i), hi = __shfl_sync(0xFFFFFFFFu, scale, 16 + block + i);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        acc[v] = fmaf((part[0][v] + part[1][v]) * x.unit(v & 1), v < 2 ? lo : hi, acc[v]);
        part[0][v] = part[1][v] = 0.f;
      }
    }
  }
  if (!kW8)   // tensor cores truncate: their sums go on for a chunk only
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(part[0][v] + part[1][v], x.unit(v & 1), acc[v]);
}

// Once read, they leave L2 first: what else lies there (the kernels' code, the tokens) stays.
__device__ __forceinline__ uint64_t read_once() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 128 bytes of 16 weight rows: [gate, up] x 8 features of an expert, or 16 outputs.
__device__ __forceinline__ void load_up(uint8_t* to, const CUtensorMap* map, int word, int f0, int e, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, "
      "%5}], [%6], %7;" ::"r"(smem_u32(to)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(word), "r"(f0), "r"(0), "r"(e), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_down(uint8_t* to, const CUtensorMap* map, int word, int d0, int e, uint64_t* bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], "
      "[%5], %6;" ::"r"(smem_u32(to)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(word), "r"(d0), "r"(e), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ int loads_of(int k, int size) { return (k * size + kCol - 1) / kCol; }

// The weights of the routed and of the shared expert, as 32-bit words.
struct Maps {
  CUtensorMap routed, shared;
};

__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return __ffs(m) - 1;
}

// Slots of up to 32 experts, one a lane with its tokens m (0: none), behind n slots and `rows` rows of a; counts them up.
__device__ __forceinline__ void add_slots(Slot* slots, int e, uint32_t m, int& n, int& rows, int lane) {
  const int own = __popc(m), parts = divide_up(own, kTokens);
  int sum = own << 16 | parts;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += o;
  }
  int at = n + (sum & 0xFFFF) - parts, base = rows + (sum >> 16) - own;
  for (int left = own; left > 0; left -= kTokens, base += kTokens) {
    const uint32_t all = m;
    for (int i = 0; i < kTokens; ++i) m &= m - 1;
    slots[at++] = {e, all ^ m, base};
  }
  const int all = __shfl_sync(0xFFFFFFFFu, sum, 31);
  n += all & 0xFFFF;
  rows += all >> 16;
}

// Slot q of the shared expert.
__device__ __forceinline__ Slot shared_slot(int q, int t) {
  return {-1, ((1u << min(kTokens, t - kTokens * q)) - 1) << (kTokens * q), kTokens * q};
}

// The slots of the picked experts, then those of the shared one; every thread of the CTA.
template <int kWarps, int kStages>
__device__ __forceinline__ void list_slots(const LayerParams& p, const Plan& P, uint8_t* smem, Shared<kWarps, kStages>& S) {
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + P.at_mask);   // zeros, as prepare() leaves them
  int* ids = reinterpret_cast<int*>(smem + P.at_ids);
  float* gates = reinterpret_cast<float*>(smem + P.at_gates);
  Slot* slots = reinterpret_cast<Slot*>(smem + P.at_slots);
  const int pairs = p.t * p.k, lane = threadIdx.x & 31;
  const bool few = pairs <= 32;   // one warp sees all pairs: slots in the order of their first ones (2.0 us -> 1.1 us)
  if (!few) {
    for (int i = threadIdx.x; i < pairs; i += 32 * kWarps) {
      const int e = __ldcg(p.ids + i);
      ids[i] = e;
      gates[i] = __ldcg(p.gates + i);
      if (e >= 0 && e < p.E) atomicOr(&mask[e], 1u << (i / p.k));
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    int n = 0, rows = 0;
    if (few) {
      const int e = lane < pairs ? __ldcg(p.ids + lane) : -1;
      if (lane < pairs) ids[lane] = e, gates[lane] = __ldcg(p.gates + lane);
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      uint32_t m = 0;
      if (e >= 0 && e < p.E && __ffs(same) - 1 == lane)
        for (uint32_t left = same; left; left &= left - 1) m |= 1u << ((__ffs(left) - 1) / p.k);
      add_slots(slots, e, m, n, rows, lane);
    } else {
      for (int e0 = 0; e0 < p.E; e0 += 32) {
        const uint32_t m = e0 + lane < p.E ? mask[e0 + lane] : 0;
        if (__any_sync(0xFFFFFFFFu, m != 0)) add_slots(slots, e0 + lane, m, n, rows, lane);
      }
    }
    const int shared = p.fs ? divide_up(p.t, kTokens) : 0;
    if (lane < shared) slots[n + lane] = shared_slot(lane, p.t);
    if (lane == 0) S.n_routed = n, S.n_slots = n + shared;
  }
  __syncthreads();
}

// What needs no input.
template <int kWarps, int kStages>
__device__ __forceinline__ void prepare(const LayerParams& p, const Maps& maps, const Plan& P, uint8_t* smem,
                                        Shared<kWarps, kStages>& S) {
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + P.at_mask);
  for (int i = threadIdx.x; i < p.E; i += 32 * kWarps) mask[i] = 0;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&S.full[w][i], 1);
    S.waits.abort = 0;
    S.waits.limit = p.limit;
    fence_mbar_init();
  } else if (threadIdx.x < 3) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(threadIdx.x == 1 || !p.fs ? &maps.routed : &maps.shared))
                 : "memory");
  }
  __syncthreads();
}

// ------------------------------------------------------------------ up

template <bool kBf16, bool kW8>
__global__ void __launch_bounds__(32 * kTeams * team_of(kW8), 1)
    k_layer_up(const __grid_constant__ Maps maps, const __grid_constant__ LayerParams p, const __grid_constant__ Plan P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int kTeam = team_of(kW8), kWarps = kTeams * kTeam, kStages = kTeamStages / kTeam;
  __shared__ Shared<kWarps, kStages> S;
  __shared__ float4 s_acc[2][kTeams][32];   // the second warps' sums, and what became of a team's waits; two units in turn
  __shared__ int s_ok[2][kTeams][kTeam];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  constexpr int kSize = kW8 ? 1 : 2;   // bytes of a weight
  constexpr int kChunk = kColsUp * kCol / kSize, kStageBytes = kColsUp * kColBytes;   // values of a chunk
  prepare(p, maps, P, smem, S);
  pdl_wait();
  pdl_trigger();
  const Slot* slots = reinterpret_cast<const Slot*>(smem + P.at_slots);
  const int per = p.f / 8, per_shared = p.fs / 8, of_shared = p.fs ? divide_up(p.t, kTokens) * per_shared : 0;
  const int mates = kTeam > 1 && p.d > kChunk ? kTeam : 1;   // units of one chunk: one warp each
  const int teams = kWarps / mates, stride = gridDim.x * teams, team = warp % teams, member = warp / teams;
  int units = of_shared;   // and the routed ones, once they are known
  uint8_t* const stages = smem + warp * kStages * kStageBytes;
  uint64_t* const full = S.full[warp];
  const uint64_t policy = read_once();

  // A place in this team's units and this warp's chunks: the shared expert's units first, which are known before the picked experts.
  struct Place {
    int unit, k0;
    Slot slot;
    int f, f0;
  };
  const auto enter = [&](Place& at) {
    at.k0 = member * kChunk;
    if (at.unit >= units) return;
    const bool shared = at.unit < of_shared;
    const int i = shared ? at.unit : at.unit - of_shared, n = shared ? per_shared : per, s = i / n;
    at.slot = shared ? shared_slot(s, p.t) : slots[s];
    at.f = shared ? p.fs : p.f;
    at.f0 = 8 * (i - s * n);
  };
  Place next;
  next.unit = blockIdx.x + team * gridDim.x;   // as many on every SM as can be
  enter(next);
  int loads = 0;
  const auto load = [&] {   // the next chunk into the next stage, which no lane reads any more
    if (next.unit >= units) return;
    if (loads < p.stall && elect_one()) {
      const int s = loads % kStages, cols = loads_of(min(kChunk, p.d - next.k0), kSize);
      mbar_arrive_expect_tx(&full[s], cols * kColBytes);
      for (int i = 0; i < cols; ++i)
        load_up(stages + s * kStageBytes + i * kColBytes, next.slot.expert < 0 ? &maps.shared : &maps.routed,
                (next.k0 * kSize + i * kCol) / 4, next.f0, max(next.slot.expert, 0), &full[s], policy);
    }
    ++loads;
    next.k0 += mates * kChunk;
    if (next.k0 >= p.d) {
      next.unit += stride;
      enter(next);
    }
  };
  for (int i = 0; i < kStages; ++i) load();
  list_slots(p, P, smem, S);
  units += S.n_routed * per;
  if (next.unit >= of_shared) enter(next);
  while (loads < kStages && next.unit < units) load();

  int it = 0, n_unit = 0;
  bool ok = true;
  Place at;
  for (at.unit = blockIdx.x + team * gridDim.x; ok && at.unit < units; at.unit += stride, ++n_unit) {
    enter(at);
    const int rows = __popc(at.slot.mask), f = at.f, f0 = at.f0;
    const float* scale = nullptr;   // lanes 0 .. 15: of the gate rows, 16 .. 31: of the up rows
    if (kW8) {
      const int kb = divide_up(p.d, 128);
      scale = (at.slot.expert < 0 ? p.shared.gate_up_scale
                                  : p.routed.gate_up_scale + static_cast<long long>(at.slot.expert) * divide_up(2 * f, 128) * kb) +
              (lane < 16 ? f0 : f + f0) / 128 * kb;
    }
    float acc[4] = {};
    const uint16_t* x = p.x + nth_bit(at.slot.mask, min(g, rows - 1)) * p.ldx;
    for (int k0 = member * kChunk; k0 < p.d; k0 += mates * kChunk, ++it) {
      const int s = it % kStages, k = min(kChunk, p.d - k0);
      TokenWords<kW8, kTokensUp> tokens;
      tokens.load(x + k0, k, lane);
      float sc = 0.f;
      if (kW8 && kCol * (lane & 15) < k) sc = __ldg(scale + k0 / 128 + (lane & 15));
      if (!(ok = wait_bar_warp(&full[s], (it / kStages) & 1, &S.waits))) break;
      chunk_products<kBf16, kW8, kTokensUp>(acc, stages + s * kStageBytes, tokens, k, sc, 0, lane);
      __syncwarp();
      load();
    }
    if (mates > 1) {   // the second warp's sums go to the first's (who writes a buffer again knows that the other came to the unit
                       // between)
      const int buf = n_unit & 1;
      if (member) s_acc[buf][team][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (lane == 0) s_ok[buf][team][member] = ok;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kTeam) : "memory");
      ok = s_ok[buf][team][0] && s_ok[buf][team][1];
      if (member) continue;
      const float4 v = s_acc[buf][team][lane];
      acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
    }
    // this lane: gate and up of one feature, columns 2 (lane % 4) and the next; the eight features of a column are the lanes that
    // differ in lane / 4
    uint16_t* a = p.a + (at.slot.expert < 0 ? static_cast<long long>(p.t) * p.k * p.f : 0LL) +
                  static_cast<long long>(at.slot.base) * f + f0 + row_of(g);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 2 * (lane & 3) + i;
      const bool there = ok && col < rows;
      constexpr bool kHalf = half_a(kBf16, kW8);
      if (!kHalf && !there) continue;
      float v = 0.f;
      if (there) {
        float gate = 1.f;
        if (at.slot.expert >= 0) {
          const int* ids = reinterpret_cast<const int*>(smem + P.at_ids);
          const float* gates = reinterpret_cast<const float*>(smem + P.at_gates);
          const int t = nth_bit(at.slot.mask, col);
          gate = 0.f;
          for (int j = 0; j < p.k; ++j) gate += ids[t * p.k + j] == at.slot.expert ? gates[t * p.k + j] : 0.f;
        }
        v = gate * (gelu16(acc[i], p.gelu) * acc[2 + i]);
      }
      uint16_t word = kHalf ? __half_as_ushort(__float2half_rn(v)) : float_to_bf16_bits(v);
      if (kHalf) {
        uint32_t top = __float_as_uint(v) & 0x7FFFFFFFu;
        uint32_t enough = __ballot_sync(0xFFFFFFFFu, top >= Packed::kSmall || !there);   // of a column: one is enough
        enough |= enough >> 16;
        enough |= enough >> 8;
        enough |= enough >> 4;
        if (__any_sync(0xFFFFFFFFu, top >= Packed::kLarge) || (enough & 15) != 15) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          const uint32_t e = Packed::exponent(top);
          const int own = Packed::integer(v, e), last = __shfl_sync(0xFFFFFFFFu, own, 28 + (lane & 3));
          if (Packed::needed(top)) word = Packed::word(row_of(g), own, last, e);
        }
      }
      if (there) a[static_cast<long long>(col) * f] = word;
    }
  }
  __syncthreads();
  if (S.waits.abort) report_and_settle(p.gave_up);
}

// ------------------------------------------------------------------ down

__device__ __forceinline__ float ld_rank(const float* at, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <bool kBf16, bool kW8>
__global__ void __launch_bounds__(32 * kWarpsDown, 2) k_layer_down(const __grid_constant__ Maps maps, const __grid_constant__ LayerParams p,
                                                         const __grid_constant__ Plan P, int split) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Shared<kWarpsDown, kStagesDown> S;
  constexpr int kWarps = kWarpsDown, kStages = kStagesDown, kThreads = 32 * kWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  const int rank = static_cast<int>(cluster_rank()), d0 = blockIdx.x / split * 16;
  constexpr int kSize = kW8 ? 1 : 2;
  constexpr int kStageBytes = kColsDown * kColBytes, kColValues = kCol / kSize;
  prepare(p, maps, P, smem, S);
  // CTAs that start after their launch gave up do nothing, or each wave of them would wait as long (asked by the warp that is the
  // last to have pairs to list: by the third one 19 tokens took 0.3 us more)
  if (tid == kThreads - 32 && *static_cast<volatile unsigned long long*>(&p.gave_up->grid) == this_grid()) {
    S.waits.abort = 2;
    atomicAdd(&p.gave_up->count, 1u);
  }
  // ids and weights are older than the first kernel, which let this one start after its own wait
  list_slots(p, P, smem, S);
  const Slot* slots = reinterpret_cast<const Slot*>(smem + P.at_slots);
  const int n_routed = S.n_routed;
  // a unit's columns of 128 bytes, slot after slot, in equal parts: a chunk lies in one slot and one part
  const int per = divide_up(p.f, kColValues), per_shared = divide_up(p.fs, kColValues);
  const int all = n_routed * per + (S.n_slots - n_routed) * per_shared;
  const int part = rank * kWarps + warp, parts = split * kWarps;
  const int first = static_cast<int>(static_cast<long long>(all) * part / parts);
  const int end = static_cast<int>(static_cast<long long>(all) * (part + 1) / parts);
  uint8_t* const stages = smem + warp * kStages * kStageBytes;
  uint64_t* const full = S.full[warp];
  const uint64_t policy = read_once();
  float* const sums = reinterpret_cast<float*>(smem + P.at_sums);   // [warp][token][16]
  float* const own = sums + warp * p.t * 16;
  for (int i = lane; i < p.t * 16; i += 32) own[i] = 0.f;

  struct Place {
    int slot, col, left;   // in the slot; of this part's columns from here on
    __device__ __forceinline__ int cols(int of_slot) const { return min(min(kColsDown, left), of_slot - col); }
  };
  const auto of_slot = [&](const Place& at) { return at.slot >= n_routed ? per_shared : per; };
  const auto advance = [&](Place& at) {
    const int n = at.cols(of_slot(at));
    at.left -= n;
    at.col += n;
    if (at.col == of_slot(at)) at.col = 0, ++at.slot;
  };
  const auto load = [&](const Place& at, int s) {
    const int cols = at.cols(of_slot(at));
    mbar_arrive_expect_tx(&full[s], cols * kColBytes);
    for (int i = 0; i < cols; ++i)
      load_down(stages + s * kStageBytes + i * kColBytes, at.slot >= n_routed ? &maps.shared : &maps.routed, (at.col + i) * (kCol / 4),
                d0, max(slots[at.slot].expert, 0), &full[s], policy);
  };
  Place at;
  at.left = S.waits.abort == 2 ? 0 : end - first;
  {
    const bool shared = first >= n_routed * per;
    const int i = shared ? first - n_routed * per : first, n = max(shared ? per_shared : per, 1), s = i / n;
    at.slot = shared ? n_routed + s : s;
    at.col = i - s * n;
  }
  const Place start = at;
  Place next = at;
  int loads = 0;
  const auto load_next = [&] {
    if (next.left <= 0 || loads >= p.stall) return;
    if (elect_one()) load(next, loads % kStages);
    ++loads;
    advance(next);
  };
  for (int i = 0; i < kStages; ++i) load_next();
  __syncwarp();
  pdl_wait();      // a; and y may be in use until here
  pdl_trigger();

  bool ok = true, odd = false;
  int it = 0;
  const int db = divide_up(p.d, 128);
  const auto add = [&](auto careful) {
    constexpr bool kCareful = decltype(careful)::value;
    constexpr int kTokenCols = tokens_down(kW8);
    constexpr bool kHalf = half_a(kBf16, kW8);
    float acc[4] = {};
    for (; at.left > 0; ++it) {
      const int s = it % kStages, k0 = at.col * kColValues;
      const bool shared = at.slot >= n_routed;
      const Slot slot = slots[at.slot];
      const int f = shared ? p.fs : p.f, k = min(at.cols(of_slot(at)) * kColValues, f - k0);
      const uint16_t* a = p.a + (shared ? static_cast<long long>(p.t) * p.k * p.f : 0LL) +
                          static_cast<long long>(slot.base + min(g, __popc(slot.mask) - 1)) * f + k0;
      std::conditional_t<kCareful, ScaledWords<kW8, kTokenCols>, TokenWords<kW8, kTokenCols>> tokens;
      tokens.load(a, k, lane);
      float sc = 0.f;
      if (kW8 && kCol * (lane & 15) < k) {
        const long long block = (shared ? 0LL : static_cast<long long>(slot.expert) * db) + d0 / 128;
        sc = __ldg((shared ? p.shared.down_scale : p.routed.down_scale) + block * divide_up(f, 128) + k0 / 128 + (lane & 15));
      }
      if (!(ok = wait_bar_warp(&full[s], (it / kStages) & 1, &S.waits))) break;
#pragma unroll
      for (int c = 0; c < kColsDown; c += kTokenCols) {
        const int done = c * kColValues;
        if (c) {
          if (done >= k) break;
          tokens.load(a + done, k - done, lane);
        }
        if constexpr (kCareful) tokens.scale(lane);
        chunk_products<!kHalf, kW8, kTokenCols>(acc, stages + s * kStageBytes + c * kColBytes, tokens, k - done, sc, c, lane);
      }
      __syncwarp();
      load_next();
      const int was = at.slot;
      advance(at);
      if (at.slot != was || at.left <= 0) {   // two rows of columns 2 (lane % 4) and the next
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int col = 2 * (lane & 3) + (v & 1);
          if (col < __popc(slot.mask)) own[nth_bit(slot.mask, col) * 16 + row_of(g) + 8 * (v >> 1)] += acc[v];
          odd |= isnan(acc[v]);
          acc[v] = 0.f;
        }
      }
    }
  };
  add(std::false_type{});
  // fp16: sums that are NaN may have met packed values; once more, with care (asked of every chunk's values beforehand, or with the
  // care in the same loop, that is 3 to 5 % of the layer)
  if (half_a(kBf16, kW8) && ok && __any_sync(0xFFFFFFFFu, odd)) {
    at = next = start;
    __syncwarp();
    for (int i = lane; i < p.t * 16; i += 32) own[i] = 0.f;
    for (int i = 0; i < kStages; ++i) load_next();
    __syncwarp();
    add(std::true_type{});
  }
  __syncthreads();
  // the warps' sums; each CTA's are then in the first warp's place
  for (int i = tid; i < 16 * p.t; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[v * p.t * 16 + i];
    sums[i] = sum;
  }
  ok = !S.waits.abort;
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (ok)
    for (int i = tid; i < 16 * p.t; i += kThreads) {
      const int col = i >> 4, row = i & 15;
      if (col % split != rank) continue;
      float sum = sums[i];
      if (split > 1) {   // all on their way at once
        float v[kMostSplit];
#pragma unroll
        for (int r = 0; r < kMostSplit; ++r) v[r] = r < split ? ld_rank(sums + i, r) : 0.f;
        sum = 0.f;
#pragma unroll
        for (int r = 0; r < kMostSplit; ++r) sum += v[r];
      }
      const long long to = col * p.ldy + d0 + row;
      if (p.out_f32)
        static_cast<float*>(p.y)[to] = sum;
      else
        static_cast<uint16_t*>(p.y)[to] = kBf16 ? float_to_bf16_bits(sum) : __half_as_ushort(__float2half_rn(sum));
    }
  if (split > 1) cluster_sync();   // the others may still read this CTA's sums
  __syncthreads();
  if (S.waits.abort == 1) report_and_settle(p.gave_up);
}

// ------------------------------------------------------------------ launches

// Of the routed experts: each has a token at least, or eight.
int most_slots(const LayerParams& p) { return std::min(p.t * p.k, p.E + p.t * p.k / kTokens); }

Plan make_plan(const LayerParams& p, bool down) {
  Plan P{};
  const int slots = most_slots(p) + divide_up(p.t, kTokens);
  P.at_sums = (down ? kWarpsDown * kStagesDown * kColsDown : kTeams * kTeamStages * kColsUp) * kColBytes;
  P.at_mask = P.at_sums + (down ? kWarpsDown * p.t * 64 : 0);
  P.at_ids = P.at_mask + 4 * p.E;
  P.at_gates = P.at_ids + 4 * p.t * p.k;
  P.at_slots = P.at_gates + 4 * p.t * p.k;
  P.bytes = P.at_slots + static_cast<int>(sizeof(Slot)) * slots + 1024;   // the stages start at a multiple of 1024
  return P;
}

bool encode_words(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                  const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dim, stride,
                          box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [E][2][f][d] in boxes of 128 bytes x 8 features x both halves.
bool map_up(CUtensorMap* m, const void* base, int E, int f, int d, int size) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * size;
  const cuuint64_t dim[4] = {row / 4, static_cast<cuuint64_t>(f), 2, static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[3] = {row, row * f, row * 2 * f};
  const cuuint32_t box[4] = {kCol / 4, 8, 2, 1};
  return encode_words(m, base, 4, dim, stride, box);
}

// [E][d][f] in boxes of 128 bytes x 16 outputs.
bool map_down(CUtensorMap* m, const void* base, int E, int d, int f, int size) {
  const cuuint64_t row = static_cast<cuuint64_t>(f) * size;
  const cuuint64_t dim[3] = {row / 4, static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[2] = {row, row * d};
  const cuuint32_t box[3] = {kCol / 4, 16, 1};
  return encode_words(m, base, 3, dim, stride, box);
}

template <typename K, typename... A>
bool launch(K kernel, int grid, int threads, const Plan& P, int cluster, cudaStream_t s, const A&... args) {
  if (!allow_smem(kernel, kMostSmem)) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = P.bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <bool kBf16, bool kW8>
bool launch_both(const LayerParams& p, int sms, cudaStream_t s) {
  constexpr int kSize = kW8 ? 1 : 2;
  const Plan up = make_plan(p, false), down = make_plan(p, true);
  Maps m_up, m_down;
  if (!map_up(&m_up.routed, p.routed.gate_up, p.E, p.f, p.d, kSize) ||
      !map_down(&m_down.routed, p.routed.down, p.E, p.d, p.f, kSize))
    return false;
  if (p.fs && (!map_up(&m_up.shared, p.shared.gate_up, 1, p.fs, p.d, kSize) ||
               !map_down(&m_down.shared, p.shared.down, 1, p.d, p.fs, kSize)))
    return false;
  // one CTA an SM, or as many as the units of the most slots need; a CTA's teams share the units evenly
  const int slots = most_slots(p);
  const long long units = static_cast<long long>(slots) * (p.f / 8) + divide_up(p.t, kTokens) * (p.fs / 8);
  const int grid = static_cast<int>(std::min<long long>(sms, units));
  if (!launch(k_layer_up<kBf16, kW8>, grid, 32 * kTeams * team_of(kW8), up, 1, s, m_up, p, up)) return false;
  const int blocks = p.d / 16, cols = slots * divide_up(p.f * kSize, kCol) + divide_up(p.fs * kSize, kCol);
  int split = 1;
  // Up to two CTAs an SM (16 experts of f = 2048, 4 tokens: d = 1024 split in 4 31.1 us, in 2 33.8; d = 512 in 4 21.6, in 1 31.8),
  // but of eight only as many as SMs: two an SM do not all start at once (d = 512 in 8 26.3; d = 256 in 8 16.7, in 4 18.3).
  while (split < kMostSplit && 2 * split * blocks <= (split < 4 ? 2 : 1) * sms && 2 * split * kWarpsDown * kColsDown <= cols) split *= 2;
  return launch(k_layer_down<kBf16, kW8>, blocks * split, 32 * kWarpsDown, down, split, s, m_down, p, down, split);
}

}  // namespace

bool launch_layer(bool weights8, const LayerParams& params, cudaStream_t s) {
  LayerParams p = params;
  const WaitLimits l = wait_limits();
  p.limit = l.cycles1024, p.stall = l.loads;
  if (!(p.gave_up = gave_up_here())) return false;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  if (weights8) return p.bf16 ? launch_both<true, true>(p, sms, s) : launch_both<false, true>(p, sms, s);
  return p.bf16 ? launch_both<true, false>(p, sms, s) : launch_both<false, false>(p, sms, s);
}

}  // namespace moe

