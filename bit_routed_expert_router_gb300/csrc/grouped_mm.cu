// 16-bit products grouped by expert with ragged sizes, on tcgen05.
//
//   forward     y[r, n]     = sum_k W[e][n, k] x[r, k]          rows r of expert e
//   gradient    dx[r, k]    = sum_n W[e][n, k] dy[r, n]
//   weights     dW[e][n, k] = sum_{r of e} dy[r, n] x[r, k]
//
// bf16 or fp16 operands, fp32 accumulators in tensor memory, one rounding at
// the store.  The weights' features are the MMA's M side and the rows its N
// side, so a ragged group costs its rows rounded up to 32 (16 in the small
// kernel) instead of to a tile of 128 or 256: an expert's rows are cut into
// equal parts of at most 256 and each part's N is set per instruction.
//
// k_grouped: persistent, pairs of CTAs (one CTA per SM), each with tiles in
// turn or taken as it gets done (Walk).  A pair computes 256 features x up to
// 256 rows with cta_group::2 MMAs; each CTA stages its 128 features and half of
// the rows, so a staged byte feeds twice the products that it would in a lone
// CTA.  Two accumulators of 256 columns: the epilogue of one tile overlaps the
// next tile's products.  Roles: warp 0 loads, warp 1 of the even CTA issues,
// warps 2-9 store; in weight gradients warp 10 clears the rows behind a group's
// end in the last stage, with adapters warps 10-13 write u and warp 14 lists
// the adapters.  The loading and issuing threads are elected (elect.sync): with
// lane == 0 in its place an MMA took 170 cycles whatever its N, against 135 for
// N = 256 and 87 for N = 160.
//
// k_grouped_small: few rows per expert (decode).  The weights are read once
// and nothing else matters, so a CTA takes 128 features x up to 64 rows, the
// reduction split over a cluster whose CTAs add their accumulators through
// distributed shared memory in rank order (no atomics, no workspace).
#include <algorithm>
#include <atomic>
#include <limits>
#include <map>
#include <mutex>
#include <type_traits>

#include "gelu16.cuh"
#include "grouped.h"
#include "tc16.cuh"
#include "tensor_map.h"

namespace moe {

namespace {

using namespace tc16;

// CTAs that gave up on this device, and the number of the last one's grid (plus
// one; the replays of a graph's node share theirs).  The count is never taken
// back: each stream that asks compares it with what it was told before.
__device__ uint32_t g_gave_up;
__device__ unsigned long long g_gave_up_grid;

constexpr int kMaxE = 1024;
constexpr int kStageBytes = 32768;   // 128 features x 64 and up to 128 columns x 64, 16 bits
constexpr int kHalf = 16384;
constexpr int kEpiPitch = 80;        // bytes between staged rows of 64 and of 32 bytes: multiples of 16, and the
constexpr int kEpiPitch16 = 48;      // 16-byte words of eight rows hit all 32 banks
constexpr int kEpiWarps = 8;         // two for each quarter of the tensor-memory lanes, 32 columns in turn
constexpr int kEpiBytes = 4 * 16 * kEpiPitch16;
constexpr int kUWarps = 4;           // adapters: warps that stage u
constexpr int kAccCols = 256;
// k64 steps that are summed in one accumulator.  The MMA adds its products to the accumulator with truncation, so a sum of
// products of one sign falls short by about 6e-9 of itself a product (measured: 4e-4 at 65,536 products, 10 % at 2^24);
// longer reductions go in pieces, which the warps that read them add with rounding.  fp32 outputs in pieces of 384 products
// (2816 products of either sign: relative error 2.6e-6 in one accumulator, 3.5e-7 in pieces); 16-bit outputs in pieces of
// 4096, short by at most 2.5e-5 where their own rounding is half a step of 4.9e-4 (fp16) or 3.9e-3 (bf16).
constexpr int kSegSteps = 6, kLongSteps = 64;

// The weight gradient's tiles have few stages each and store far more than they
// load: two buffers a warp for TMA stores, and a stage less.
template <int kMode, int kEpi>
struct BigCfg {
  static constexpr int kStages = kMode == GM_WGRAD ? 5 : 6;
  static constexpr int kEpiBytes = kMode == GM_WGRAD ? 4096 : kEpi == GM_ADAPT ? 4 * 8 * kEpiPitch : moe::kEpiBytes;
  static constexpr int kThreads = 32 * (2 + kEpiWarps + (kEpi == GM_ADAPT ? kUWarps + 1 : kMode == GM_WGRAD ? 1 : 0));
};

constexpr int kLists = 4;
struct AdaptSmem {
  int id[kLists][256];     // adapter of each column of a tile, -1 for none (tiles in turn)
  int list[kLists][256];   // its distinct adapters, in order
  int n_list[kLists];
  // A value of the tile's B rows is not finite.  Sixteen tiles in turn: a tile is listed (and its mark cleared) at most
  // kLists tiles ahead of the loads, which run at most kStages steps, so as many tiles, ahead of the products, and these
  // two ahead of the stores.
  volatile int broken[16];
  uint64_t u_full[8], list_full[kLists], list_empty[kLists];
};
struct NoSmem {};

// fp32 weight gradients: the answers to a pair's requests for the next tile, in turn.
// kAhead at a time: the tile at hand and as many more are the pair's (one: 381 us, two 375, five 377).
constexpr int kAnswers = 8, kAhead = 2;
template <int kMode, int kEpi>
constexpr bool kTakes = kMode == GM_WGRAD && kEpi == GM_F32;   // (see Walk)
struct TakeSmem {
  alignas(16) uint8_t answer[kAnswers][16];
  uint64_t full[kAnswers], empty[kAnswers];
};

// A CTA's bounded waits.
struct Waits {
  volatile int abort;   // 1: one ran out; 2: the launch had given up before this CTA started
  int limit;            // of each, in 1024 cycles
};

template <int kMode, int kEpi>
struct BigSmem {
  static constexpr int kStages = BigCfg<kMode, kEpi>::kStages;
  uint8_t stage[kStages][kStageBytes];
  alignas(1024) uint8_t epi[kEpiWarps][BigCfg<kMode, kEpi>::kEpiBytes];
  uint64_t full[kStages], empty[kStages], tail[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  Waits waits;
  std::conditional_t<kTakes<kMode, kEpi>, TakeSmem, NoSmem> take;
  std::conditional_t<kEpi == GM_ADAPT, AdaptSmem, NoSmem> ad;
  int off[(kEpi == GM_ADAPT ? 1 : kMaxE) + 1];    // clamped to [0, m]
  int tiles[(kEpi == GM_ADAPT ? 1 : kMaxE) + 1];  // column tiles before each expert
};
static_assert(sizeof(BigSmem<GM_FWD, GM_PLAIN>) + 1024 <= 227 * 1024 &&
                  sizeof(BigSmem<GM_FWD, GM_ADAPT>) + 1024 <= 227 * 1024 &&
                  sizeof(BigSmem<GM_WGRAD, GM_PLAIN>) + 1024 <= 227 * 1024,
              "one CTA per SM");
static_assert(kEpiBytes >= 4 * 8 * kEpiPitch && kEpiBytes % 16 == 0 &&
                  kEpiPitch % 16 == 0 && kEpiPitch16 % 16 == 0,
              "staged rows");

__device__ __forceinline__ unsigned long long this_grid() {
  unsigned long long g;
  asm volatile("mov.u64 %0, %%gridid;" : "=l"(g));
  return g + 1;
}

constexpr long long kSettleCycles = 20000000;

// Bounded wait that also ends when another role of the CTA gave up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Waits* w) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (w->abort) return false;
    if (clock64() - t0 > 1024LL * w->limit) {
      w->abort = 1;
      return false;
    }
  }
}

// The same by a whole warp, which then agrees on the outcome.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, Waits* w) {
  return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, w));
}

// The end of a CTA that gave up, by all of its threads.  Copies, products and
// arrivals may be on their way, and no barrier tells which: those of a pair's odd
// CTA count on the even one's barriers, of which the phases that miss a share
// stay open.  All of them take microseconds; the CTA keeps its memories for
// another 10 ms.
__device__ __forceinline__ void report_and_settle() {
  if (threadIdx.x == 0) {
    *static_cast<volatile unsigned long long*>(&g_gave_up_grid) = this_grid();
    atomicAdd(&g_gave_up, 1u);
  }
  const long long t0 = clock64();
  while (clock64() - t0 < kSettleCycles) __nanosleep(1000);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Row range of expert e: inside [0, m] whatever the offsets hold.
__device__ __forceinline__ int clamp_off(int v, int m) { return min(max(v, 0), m); }

// The two operands' tensor maps.  The rows' map comes in boxes of 16 (i + 1)
// rows, so a stage's rows are one load whatever their number: loads of 16 rows
// each kept the whole kernel at 237 us where the weights alone take 157 (gate/up
// input gradient, 32,768 rows).
constexpr int kRowMaps = 8;
struct GmMaps {
  CUtensorMap a;
  CUtensorMap c;   // adapters: their B; weight gradient: the output
  CUtensorMap b[kRowMaps];
};

struct Tile {
  int e, f0;         // expert, first feature
  int c0, cols, n;   // first column (a row of x, or of this expert's gradient), columns, columns rounded up for the MMA
  int row0, rows;    // GM_WGRAD: the expert's rows
  int steps;         // k64 steps
};

// Tile t of the launch in the order expert, feature tile, column tile: the
// pairs that run together share an expert's rows and weights through L2.
template <int kMode, int kFeat, typename Smem>
__device__ __forceinline__ bool tile_at(const Smem& S, const GmParams& p, int t, int& e, Tile& T) {
  const int ft = (p.feat + kFeat - 1) / kFeat;
  if constexpr (kMode == GM_WGRAD) {
    const int ct = (p.cols + 255) / 256, per = ft * ct;
    e = t / per;
    if (e >= p.E) return false;
    const int rem = t - e * per, c = rem / ft;
    T.e = e;
    T.f0 = (rem - c * ft) * kFeat;
    T.c0 = c * 256;
    T.cols = min(256, p.cols - T.c0);
    T.n = 256;
    T.row0 = S.off[e];
    T.rows = max(S.off[e + 1] - T.row0, 0);
    T.steps = (T.rows + 63) / 64;
    return true;
  } else {
    while (e < p.E && S.tiles[e + 1] * ft <= t) ++e;
    if (e >= p.E) return false;
    const int nt = S.tiles[e + 1] - S.tiles[e], rem = t - S.tiles[e] * ft, f = rem / nt, c = rem - f * nt;
    const int lo = S.off[e], rows = S.off[e + 1] - lo;
    const int width = ((rows + nt - 1) / nt + 31) & ~31;
    T.e = e;
    T.f0 = f * kFeat;
    T.c0 = lo + c * width;
    T.cols = min(width, lo + rows - T.c0);
    T.n = max((T.cols + 31) & ~31, 32);   // an MMA has columns whatever the parts are
    T.row0 = T.rows = 0;
    T.steps = (p.red + 63) / 64;
    return true;
  }
}

// The tiles of a pair: its share in turn, or (fp32 weight gradients) the launch
// has a cluster for each tile and a pair that is done takes over the next one
// that has not started.  Ordinary stores are not equally fast on every SM, and
// experts differ in rows: 128 experts of 1408 x 2816 at 4 rows each 339 us in
// turn against 283, at 64 387 / 321, at 256 421 / 361.  TMA
// stores of 16 bits gain nothing (4 rows 164 / 181, 256 rows 243 / 245: the
// answer is read in the storing warps' chain), nor do the rows' products
// (32,768 rows: down 125 / 128, input gradient 221 / 224).  Taking several
// tiles at once writes pages that lie apart (two: 358 -> 367).
struct Walk {
  int t;        // tile
  uint32_t n;   // answers read
};

// The next tile.  kWarp: called by a whole warp.  `ask` runs before an answer
// is waited for; a reader gives the answer's place back at `lead_empty` (0: it
// is the asking thread itself).
template <bool kTake, bool kWarp, typename Smem, typename Ask>
__device__ __forceinline__ bool next_tile(Smem& S, Walk& w, uint32_t lead_empty, Ask ask) {
  if constexpr (kTake) {
    ask();
    if (w.t < 0) {
      w.t = blockIdx.x >> 1;
      return true;
    }
    const int s = w.n % kAnswers;
    const uint32_t parity = (w.n / kAnswers) & 1;
    if (!(kWarp ? wait_bar_warp(&S.take.full[s], parity, &S.waits) : wait_bar(&S.take.full[s], parity, &S.waits)))
      return false;
    ++w.n;
    const int block = taken_block(smem_u32(S.take.answer[s]));
    if (lead_empty) {
      fence_proxy_async_smem();
      if (kWarp) __syncwarp();
      if (!kWarp || (threadIdx.x & 31) == 0) arrive_cluster(lead_empty + 8 * s);
    }
    w.t = block >> 1;
    return block >= 0;
  } else {
    w.t += gridDim.x >> 1;
    return true;
  }
}

// ------------------------------------------------------------------ adapter term of the epilogue

// Two fp32 values in one register pair, and d = a b + d on both at once.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ void fma_f32x2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// Eight 16-bit values as four pairs of floats.
__device__ __forceinline__ void widen8(uint64_t (&o)[4], uint4 v, int bf16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = bf16 ? pack_f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                : pack_f32x2(half_lo(w[i]), half_hi(w[i]));
}

// Eight floats of u.
__device__ __forceinline__ void load_u8(uint64_t (&o)[4], const float* u) {
  asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(o[0]), "=l"(o[1]), "=l"(o[2]), "=l"(o[3]) : "l"(u));
}

// ---- the adapters' term in the persistent kernel
//
// y = W x + B_i u is a longer reduction: among the k64 steps of W and x come
// steps whose features' operand is B_i and whose columns' operand is u, zero in
// the rows of other adapters; one pair of steps (B_i is loaded once, one handshake
// for both) for each distinct adapter of the tile's rows and 64 ranks.  These
// products are of bf16 values whatever the call's type, so that u keeps fp32's
// range (as fp16 it lost bits below 2^-9 and everything past 65504): u is a value
// and its remainder, good to 2^-17, and so is fp16's B, whose eleven bits they
// hold; the product of the two remainders, 2^-15 at most, is left out.  The split
// and the third product take fp16 calls from 89 to 104 us (4096 rows in runs of 41,
// rank 64; bf16 86) and from 57 to 58 (one adapter).
// One warp of each CTA lists the tiles' adapters; four write u's steps and look
// through the B rows that TMA loaded for them: a value that is not finite would
// reach every column (0 times infinity), so it is cleared and the tile marked,
// and the storing warps add its rows' terms where they belong.  (As mma.sync products in the
// epilogue the term took the kernel from 45 to 115 us at 4096 rows and rank 64,
// since they wait for the tcgen05 products; on the ordinary pipes 145, bound by
// broadcast loads.)

// The pairs are spread over the tile's reduction, so that the warps that write
// them have the steps between for it: pair i of n comes before base step
// pair_at(i, n).
__device__ __forceinline__ int pair_at(int i, int n, int steps) { return max(1, (i + 1) * steps / (n + 1)); }

// True if one of the 16-bit values of v is infinite or NaN (all exponent bits set).
__device__ __forceinline__ uint32_t not_finite(uint32_t v, int bf16) {
  const uint32_t mask = bf16 ? 0x7F807F80u : 0x7C007C00u, one = bf16 ? 0x00800080u : 0x04000400u;
  return ((v & mask) + one) & 0x80008000u;
}

// B's row times u in fp32 if the row has a value that is not finite (an infinity or NaN then), else 0.
__device__ __noinline__ float broken_value(const uint16_t* b, const float* u, int rank, int bf16) {
  uint32_t bad = 0;
  float sum = 0.f;
  for (int k = 0; k < rank; k += 2) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(b + k));
    const float2 v = __ldcg(reinterpret_cast<const float2*>(u + k));
    bad |= not_finite(w, bf16);
    sum = fmaf(bf16 ? __uint_as_float(w << 16) : half_lo(w), v.x, sum);
    sum = fmaf(bf16 ? __uint_as_float(w & 0xFFFF0000u) : half_hi(w), v.y, sum);
  }
  return bad ? sum : 0.f;
}

// Columns row0 .. and this warp's 32 features of a marked tile: the terms that are not finite.
__device__ __forceinline__ void add_broken(float (&v)[2][16], const GmParams& p, int row0, int cols, int f0, int lane) {
  pdl_wait();   // u
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 8 * j + 2 * (lane & 3) + (i & 1);
      const int id = c < cols ? p.ids[row0 + c] : -1;
      if (id < 0 || id >= p.n_adapters) continue;
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        const int f = f0 + 16 * mb + 8 * (i >> 1) + (lane >> 2);
        if (f < p.feat)
          v[mb][4 * j + i] += broken_value(p.b + (static_cast<size_t>(id) * p.feat + f) * p.rank,
                                           p.u + static_cast<size_t>(row0 + c) * p.rank, p.rank, p.bf16);
      }
    }
}

// The upper halves of two fp32 values: them as bf16, cut off.
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// Eight values of u as bf16, and what that leaves.  `odd` turns NaN if a remainder is (that of an infinity).
__device__ __forceinline__ void split_u(const uint64_t (&u)[4], uint4& hi, uint4& lo, float& odd) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[2 * i] = __uint_as_float(static_cast<uint32_t>(u[i])), v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(u[i] >> 32));
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack16(v[2 * i], v[2 * i + 1], 1);
    const float l0 = v[2 * i] - __uint_as_float(h[i] << 16), l1 = v[2 * i + 1] - __uint_as_float(h[i] & 0xFFFF0000u);
    l[i] = pack16(l0, l1, 1);
    odd = fmaf(l0, 0.f, fmaf(l1, 0.f, odd));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// lo without the halves whose hi is not finite.
__device__ __forceinline__ uint32_t drop_odd(uint32_t hi, uint32_t lo) { return lo & ~((not_finite(hi, 1) >> 15) * 0xFFFFu); }

// Eight fp16 values as bf16: their first eight bits, and the three that these leave.  False if one is not finite.
__device__ __forceinline__ bool split_f16(const uint4& v, uint4& hi, uint4& lo) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
  __half2 odd = __half2half2(__ushort_as_half(0));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = in[i] & 0xFFF8FFF8u;
    const __half2 left = __hsub2(*reinterpret_cast<const __half2*>(&in[i]), *reinterpret_cast<const __half2*>(&top));
    odd = __hfma2(left, __half2half2(__ushort_as_half(0)), odd);   // NaN if a remainder is
    h[i] = upper_halves(half_lo(top), half_hi(top));
    l[i] = upper_halves(__low2float(left), __high2float(left));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  return (*reinterpret_cast<const uint32_t*>(&odd) & 0x7FFF7FFFu) == 0;
}

// ------------------------------------------------------------------ the persistent kernel

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}

// The stores of one warp: 32 columns of its accumulator lanes as fragments,
// turned through the warp's own shared memory so that every lane stores 16
// bytes.  All of a tensor's fragments are staged before the first is read
// back: one warp barrier each way, and four independent loads and stores.

// 32 features x 32 columns of 16-bit values: 64 contiguous bytes of a column.
__device__ __forceinline__ void store_32x32(uint32_t buf, const float (&v)[2][16], int bf16, uint16_t* out, long long ld,
                                            int cols, int feats, int lane) {
  __syncwarp();   // earlier reads of this buffer are done
#pragma unroll
  for (int j = 0; j < 4; ++j)
    stmatrix4_trans(buf + j * 8 * kEpiPitch + (lane & 7) * kEpiPitch + (lane >> 3) * 16,
                    pack16(v[0][4 * j], v[0][4 * j + 1], bf16), pack16(v[0][4 * j + 2], v[0][4 * j + 3], bf16),
                    pack16(v[1][4 * j], v[1][4 * j + 1], bf16), pack16(v[1][4 * j + 2], v[1][4 * j + 3], bf16));
  __syncwarp();
  const int f = 8 * (lane & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 8 * j + (lane >> 2);
    const uint4 w = lds128(buf + c * kEpiPitch + (lane & 3) * 16);
    if (c < cols && f < feats) *reinterpret_cast<uint4*>(out + c * ld + f) = w;
  }
}

// One feature a lane of 32 fp32 columns: each store of the warp is 128 contiguous bytes of a column.
__device__ __forceinline__ void store_f32(const float (&v)[32], float* out, long long ld, int cols, int feats, int lane) {
  if (lane >= feats) return;
  float* y = out + lane;
  if (cols >= 32) {
#pragma unroll
    for (int c = 0; c < 32; ++c) y[c * ld] = v[c];
  } else {
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < cols) y[c * ld] = v[c];
  }
}

// The weight gradient's stores: swizzled rows of 32 features in one of two
// buffers, which the TMA engine writes out while the other is filled.  A
// 64-byte segment of each column per warp and ordinary store kept the LSU's
// data pipe at 66% and the kernel at 138 us (507 MB of fp16).
__device__ __forceinline__ void tma_store_32x32(uint32_t buf, const float (&v)[2][16], const GmParams& p,
                                                const CUtensorMap* map, int f0, int c0, int e, int lane, bool lead,
                                                uint32_t& n_stores) {
  const uint32_t at = buf + 2048 * (n_stores++ & 1);
  if (lead) store_wait<1>();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 8 * j + (lane & 7);
    stmatrix4_trans(at + 64 * c + 16 * ((lane >> 3) ^ ((c >> 1) & 3)), pack16(v[0][4 * j], v[0][4 * j + 1], p.bf16),
                    pack16(v[0][4 * j + 2], v[0][4 * j + 3], p.bf16), pack16(v[1][4 * j], v[1][4 * j + 1], p.bf16),
                    pack16(v[1][4 * j + 2], v[1][4 * j + 3], p.bf16));
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lead) store_3d(map, at, f0, c0, e);
}

// 16 features x 32 columns of 16-bit values (one 16-row block): staged here ...
__device__ __forceinline__ void stage_16x32(uint32_t buf, const float (&v)[16], int bf16, int lane) {
  const int blk = lane >> 3;   // blocks: (fragment j, features 0-7), (j, 8-15), (j + 1, 0-7), (j + 1, 8-15)
#pragma unroll
  for (int j = 0; j < 4; j += 2)
    stmatrix4_trans(buf + (8 * j + (blk >> 1) * 8 + (lane & 7)) * kEpiPitch16 + (blk & 1) * 16,
                    pack16(v[4 * j], v[4 * j + 1], bf16), pack16(v[4 * j + 2], v[4 * j + 3], bf16),
                    pack16(v[4 * j + 4], v[4 * j + 5], bf16), pack16(v[4 * j + 6], v[4 * j + 7], bf16));
}

// ... and stored: 32 contiguous bytes of a column.
__device__ __forceinline__ void store_16x32(uint32_t buf, uint16_t* out, long long ld, int cols, int feats, int lane) {
  const int f = 8 * (lane & 1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = 16 * i + (lane >> 1);
    const uint4 w = lds128(buf + c * kEpiPitch16 + (lane & 1) * 16);
    if (c < cols && f < feats) *reinterpret_cast<uint4*>(out + c * ld + f) = w;
  }
}

template <int kMode, int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(BigCfg<kMode, kEpi>::kThreads, 1)
    k_grouped(const __grid_constant__ GmMaps maps, GmParams p) {
  constexpr bool kTa = kMode != GM_FWD, kTb = kMode == GM_WGRAD;
  constexpr int kFeat = kEpi == GM_GATED ? 128 : 256;   // features of a pair's tile
  constexpr bool kTake = kTakes<kMode, kEpi>;
  extern __shared__ uint8_t smem_raw[];
  using Smem = BigSmem<kMode, kEpi>;
  constexpr int kStages = Smem::kStages;
  Smem& S = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();

  if (tid == 0) {
    prefetch_map(&maps.a);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], kMode == GM_WGRAD ? 2 : 1);
      mbar_init(&S.empty[i], 1);
      mbar_init(&S.tail[i], kEpi == GM_ADAPT ? 2 : 1);
      if constexpr (kEpi == GM_ADAPT) mbar_init(&S.ad.u_full[i], 2 * kUWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.acc_full[i], 1);
      mbar_init(&S.acc_empty[i], 2 * kEpiWarps);
    }
    if constexpr (kEpi == GM_ADAPT)
      for (int i = 0; i < kLists; ++i) {
        mbar_init(&S.ad.list_full[i], 1);
        mbar_init(&S.ad.list_empty[i], kUWarps + (rank == 0 ? 2 : 1));   // and the loading and the issuing warp
      }
    if constexpr (kTake)
      for (int i = 0; i < kAnswers; ++i) {
        mbar_init(&S.take.full[i], 1);
        mbar_init(&S.take.empty[i], 2 * (BigCfg<kMode, kEpi>::kThreads / 32 - 1));   // all but one loading, one idle warp
      }
    // a pair that gave up leaves its launch's other tiles to clusters that start after it: those do nothing, or each would
    // wait as long
    S.waits.abort = kTake && *static_cast<volatile unsigned long long*>(&g_gave_up_grid) == this_grid() ? 2 : 0;
    if (S.waits.abort) atomicAdd(&g_gave_up, 1u);
    S.waits.limit = p.limit;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<true>(&S.tmem, 2 * kAccCols);
  // with adapters only the u rows come from the previous kernel, and the products of W start on the SMs it leaves (4096
  // rows 68 -> 61 us): when this kernel may start, all CTAs of the previous one run, so the bounded waits for u last as long
  // as one of those at most (64 passes of 1024 steps with the largest sizes, tens of milliseconds)
  if (kEpi != GM_ADAPT) pdl_wait();
  pdl_trigger();
  for (int e = tid; e <= p.E; e += BigCfg<kMode, kEpi>::kThreads)
    S.off[e] = p.offsets ? clamp_off(p.offsets[e], p.m) : e * p.m;
  __syncthreads();
  if (kMode != GM_WGRAD && warp == 0) {
    // offsets that go down would count rows twice: a group starts no earlier than the one before it ends
    for (int e0 = 0, before = 0; e0 <= p.E; e0 += 32) {
      const int e = e0 + lane;
      int v = e <= p.E ? S.off[e] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = max(v, o);
      }
      v = max(v, before);
      if (e <= p.E) S.off[e] = v;
      before = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    __syncwarp();
    // Parts of at most 256 rows; of 128 or 64 where the tiles then still are one round of the pairs, which few tiles of
    // 256 would leave idle (256 rows and 2816 features: 11 tiles for 76 pairs).
    int n128 = 0, n64 = 0, width = 256;
    for (int e = lane; e < p.E; e += 32) {
      const int rows = max(S.off[e + 1] - S.off[e], 0);
      n128 += (rows + 127) / 128;
      n64 += (rows + 63) / 64;
    }
    n128 = __reduce_add_sync(0xFFFFFFFFu, n128);
    n64 = __reduce_add_sync(0xFFFFFFFFu, n64);
    const int ft = (p.feat + kFeat - 1) / kFeat, pairs = gridDim.x >> 1;
    if (n64 * ft <= pairs)
      width = 64;
    else if (n128 * ft <= pairs)
      width = 128;
    int base = 0;
    if (lane == 0) S.tiles[0] = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int c = e < p.E ? (max(S.off[e + 1] - S.off[e], 0) + width - 1) / width : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, c, d);
        if (lane >= d) c += o;
      }
      if (e < p.E) S.tiles[e + 1] = base + c;
      base += __shfl_sync(0xFFFFFFFFu, c, 31);
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised
  fence_after();
  const uint32_t tmem = S.tmem;
  uint32_t lead_take = 0;
  if constexpr (kTake) lead_take = map_rank(smem_u32(S.take.empty), 0);
  const auto no_ask = [] {};
  Walk walk{kTake ? -1 : static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1), 0};

  if (warp == 0) {
    if (elect_one()) {
      const uint32_t lead_full = map_rank(smem_u32(S.full), 0);
      uint32_t it = 0, n_tile = 0;
      int e = 0;
      Tile T;
      uint32_t asked = 0;
      const auto ask = [&] {
        if constexpr (kTake) {
          for (; rank == 0 && asked < walk.n + kAhead; ++asked) {
            const int s = asked % kAnswers;
            if (!wait_bar(&S.take.empty[s], ((asked / kAnswers) & 1) ^ 1, &S.waits)) return;
            mbar_arrive_expect_tx(&S.take.full[s], 16);
            arrive_expect_cluster(map_rank(smem_u32(&S.take.full[s]), 1), 16);
            try_take_cluster(smem_u32(S.take.answer[s]), smem_u32(&S.take.full[s]));
          }
        }
      };
      const uint32_t stall = p.stall;
      while (!S.waits.abort && it < stall && next_tile<kTake, false>(S, walk, rank == 0 ? 0 : lead_take, ask) &&
             tile_at<kMode, kFeat>(S, p, walk.t, e, T)) {
        const int half = T.n / 2;
        const uint32_t bytes = kHalf + half * 128;
        int pairs = 0, pair = 0;
        [[maybe_unused]] const int lb = n_tile++ % kLists;
        if constexpr (kEpi == GM_ADAPT) {
          if (!wait_bar(&S.ad.list_full[lb], ((n_tile - 1) / kLists) & 1, &S.waits)) break;
          pairs = S.ad.n_list[lb] * ((p.rank + 63) / 64);
        }
        for (int ks = 0; it < stall && (ks < T.steps || pair < pairs); ++ks) {
          if constexpr (kEpi == GM_ADAPT) {
            for (; pair < pairs && pair_at(pair, pairs, T.steps) <= ks; ++pair, it += 2) {
              // one load of B for both stages; the writing warps go on when it has landed and both are free
              const int s = it % kStages, s2 = (it + 1) % kStages, block = pair / S.ad.n_list[lb];
              if (!wait_bar(&S.empty[s], ((it / kStages) & 1) ^ 1, &S.waits)) break;
              mbar_arrive_expect_tx(&S.tail[s], kHalf);
              load_3d<true>(smem_u32(S.stage[s]), &maps.c, 64 * block, T.f0 + 128 * rank,
                            S.ad.list[lb][pair - block * S.ad.n_list[lb]], smem_u32(&S.tail[s]));
              if (!wait_bar(&S.empty[s2], (((it + 1) / kStages) & 1) ^ 1, &S.waits)) break;
              mbarrier_arrive(&S.tail[s]);
            }
            if (S.waits.abort) break;
            if (ks >= T.steps) continue;
          }
          const int s = it % kStages;
          if (!wait_bar(&S.empty[s], ((it / kStages) & 1) ^ 1, &S.waits)) break;
          uint32_t bar = lead_full + 8 * s;
          if (kMode == GM_WGRAD) {
            if (ks == T.steps - 1 && (T.rows & 15)) {   // warp 10 sees these bytes first
              bar = smem_u32(&S.tail[s]);
              mbar_arrive_expect_tx(&S.tail[s], bytes);
            } else {
              arrive_expect_cluster(bar, bytes);
            }
          } else if (rank == 0) {
            mbar_arrive_expect_tx(&S.full[s], 2 * bytes);
          }
          const uint32_t a = smem_u32(S.stage[s]), b = a + kHalf;
          if (kMode == GM_WGRAD) {
            const int row = T.row0 + 64 * ks;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              load_2d<true>(a + 8192 * i, &maps.a, T.f0 + 128 * rank + 64 * i, row, bar);
              load_2d<true>(b + 8192 * i, &maps.b[0], T.c0 + 128 * rank + 64 * i, row, bar);
            }
          } else {
            if (kEpi == GM_GATED) {
              load_5d<true>(a, &maps.a, 64 * ks, 0, 0, (T.f0 + 64 * static_cast<int>(rank)) / 16, T.e, bar);
            } else if (kMode == GM_FWD) {
              load_3d<true>(a, &maps.a, 64 * ks, T.f0 + 128 * rank, T.e, bar);
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                load_3d<true>(a + 8192 * i, &maps.a, T.f0 + 128 * rank + 64 * i, 64 * ks, T.e, bar);
            }
            load_2d<true>(b, &maps.b[half / 16 - 1], 64 * ks, T.c0 + rank * half, bar);
          }
          ++it;
        }
        if constexpr (kEpi == GM_ADAPT) mbarrier_arrive(&S.ad.list_empty[lb]);
      }
      if constexpr (kTake)   // the answers asked for ahead of the refusal come before the pair leaves
        for (uint32_t i = walk.n; i < walk.n + kAhead - 1; ++i)
          if (!wait_bar(&S.take.full[i % kAnswers], (i / kAnswers) & 1, &S.waits)) break;
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      constexpr int kPiece = kEpi == GM_F32 ? kSegSteps : kLongSteps;
      uint32_t it = 0, count = 0, fulls = 0, us = 0;   // count: accumulators; fulls, us: phases seen, by stage
      [[maybe_unused]] uint32_t n_tile = 0;
      int e = 0;
      bool ok = true;
      Tile T;
      while (ok && next_tile<kTake, false>(S, walk, lead_take, no_ask) && tile_at<kMode, kFeat>(S, p, walk.t, e, T)) {
        if (T.steps == 0) continue;
        int buf = count & 1;
        ok = wait_bar(&S.acc_empty[buf], ((count >> 1) & 1) ^ 1, &S.waits);
        fence_after();
        uint32_t d = tmem + buf * kAccCols;
        const uint32_t idesc = instr_desc(p.bf16, 256, T.n, kTa, kTb), idesc_u = instr_desc(true, 256, T.n, kTa, kTb);
        const int red = kMode == GM_WGRAD ? T.rows : p.red;
        // stages of the operands, k of their 64
        const auto multiply = [&](int sa, int sb, int k, uint32_t idesc, bool first_step) {
          const uint64_t da = tile_desc<kTa>(smem_u32(S.stage[sa])), db = tile_desc<kTb>(smem_u32(S.stage[sb]) + kHalf);
          const int nk = (min(64, k) + 15) / 16;
          for (int kk = 0; kk < nk; ++kk)
            mma<true>(d, da + kk * kStep16<kTa>, db + kk * kStep16<kTb>, idesc, !first_step || kk != 0);
        };
        int pairs = 0, pair = 0;
        [[maybe_unused]] const int lb = n_tile % kLists;
        if constexpr (kEpi == GM_ADAPT) {
          ok = ok && wait_bar(&S.ad.list_full[lb], (n_tile++ / kLists) & 1, &S.waits);
          pairs = ok ? S.ad.n_list[lb] * ((p.rank + 63) / 64) : 0;
        }
        for (int ks = 0; ok && (ks < T.steps || pair < pairs); ++ks) {
          if constexpr (kEpi == GM_ADAPT) {
            for (; pair < pairs && pair_at(pair, pairs, T.steps) <= ks; ++pair, it += 2) {
              const int s = it % kStages, s2 = (it + 1) % kStages, k = p.rank - 64 * (pair / S.ad.n_list[lb]);
              if (!(ok = wait_bar(&S.ad.u_full[s], (us >> s) & 1, &S.waits))) break;
              us ^= 1u << s;
              fence_after();
              multiply(s, s, k, idesc_u, false);
              multiply(s, s2, k, idesc_u, false);
              if (!p.bf16) multiply(s2, s, k, idesc_u, false);
              commit_pair(&S.empty[s], 3);
              commit_pair(&S.empty[s2], 3);
            }
            if (!ok) break;
            if (ks >= T.steps) continue;
          }
          if (ks > 0 && ks % kPiece == 0) {   // the next piece in the other accumulator
            commit_pair(&S.acc_full[buf], 3);
            ++count;
            buf = count & 1;
            d = tmem + buf * kAccCols;
            if (!(ok = wait_bar(&S.acc_empty[buf], ((count >> 1) & 1) ^ 1, &S.waits))) break;
            fence_after();
          }
          const int s = it % kStages;
          if (!(ok = wait_bar(&S.full[s], (fulls >> s) & 1, &S.waits))) break;
          fulls ^= 1u << s;
          fence_after();
          multiply(s, s, red - 64 * ks, idesc, ks % kPiece == 0);
          commit_pair(&S.empty[s], 3);
          ++it;
        }
        if constexpr (kEpi == GM_ADAPT) mbarrier_arrive(&S.ad.list_empty[lb]);
        if (ok) commit_pair(&S.acc_full[buf], 3);
        ++count;
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    const int q = warp & 3;   // the tensor-memory lanes this warp may read
    const uint32_t buf16 = smem_u32(S.epi[warp - 2]);
    const uint32_t lead_empty = map_rank(smem_u32(S.acc_empty), 0);
    const bool lead = kMode == GM_WGRAD && kEpi == GM_PLAIN && elect_one();
    uint32_t count = 0, n_stores = 0;
    [[maybe_unused]] uint32_t n_tile = 0;
    int e = 0;
    Tile T;
    for (; next_tile<kTake, true>(S, walk, lead_take, no_ask) && tile_at<kMode, kFeat>(S, p, walk.t, e, T); ++n_tile) {
      // first feature of this warp's 32 lanes (GM_GATED: 16 gate and 16 up lanes of 16 features)
      const int f0 = T.f0 + (kEpi == GM_GATED ? 64 * rank + 16 * q : 128 * rank + 32 * q);
      const int feats = p.feat - f0;   // none or less: the output ends before this warp's features do
      const int c_first = 32 * ((warp - 2) >> 2);
      const long long out0 =
          (kMode == GM_WGRAD ? (static_cast<long long>(T.e) * p.cols + T.c0) : static_cast<long long>(T.c0)) * p.ldy + f0;
      if constexpr (kEpi == GM_F32) {
        // a lane holds one feature of up to 128 columns, summed over the pieces; each store of the warp is 128 contiguous
        // bytes of a column.  Read 16 columns at a time: with 32 the sums spilled, and a spilled value's way back queues
        // behind the stores (weight gradient, 512 rows an expert, 544 us against 492; sixteen storing warps 508)
        float sum[4][32];
#pragma unroll
        for (int c = 0; c < 32; ++c) sum[0][c] = sum[1][c] = sum[2][c] = sum[3][c] = 0.f;
        bool ok = true;
        for (int ks = 0; ok && ks < T.steps; ks += kSegSteps, ++count) {
          const int buf = count & 1;
          if (!(ok = wait_bar_warp(&S.acc_full[buf], (count >> 1) & 1, &S.waits))) break;
          fence_after();
          const uint32_t at = tmem + buf * kAccCols + c_first + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c_first + 64 * i < T.cols) {
#pragma unroll
              for (int c0 = 0; c0 < 32; c0 += 16) {
                float w[16];
                ld_cols16(at + 64 * i + c0, w);
#pragma unroll
                for (int c = 0; c < 16; ++c) sum[i][c0 + c] += w[c];
              }
            }
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(lead_empty + 8 * buf);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store_f32(sum[i], static_cast<float*>(p.y) + out0 + (c_first + 64 * i) * p.ldy, p.ldy, T.cols - c_first - 64 * i,
                    feats, lane);
        continue;
      }
      // 32 columns of this warp's features, rounded and stored
      const auto store = [&](float (&v)[2][16], int c0) {
        const int cols = T.cols - c0;
        if (kMode == GM_WGRAD && kEpi == GM_PLAIN) {
          tma_store_32x32(buf16, v, p, &maps.c, f0, T.c0 + c0, T.e, lane, lead, n_stores);
        } else if (kEpi == GM_GATED) {
          __syncwarp();
          if (p.h) {
            uint16_t* h = static_cast<uint16_t*>(p.h) + static_cast<long long>(T.c0 + c0) * p.ldh + f0;
            stage_16x32(buf16, v[0], p.bf16, lane);
            stage_16x32(buf16 + 32 * kEpiPitch16, v[1], p.bf16, lane);
            __syncwarp();
            store_16x32(buf16, h, p.ldh, cols, feats, lane);
            store_16x32(buf16 + 32 * kEpiPitch16, h + p.feat, p.ldh, cols, feats, lane);
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = gelu16(v[0][i], p.gelu) * v[1][i];
          stage_16x32(buf16, v[0], p.bf16, lane);
          __syncwarp();
          store_16x32(buf16, static_cast<uint16_t*>(p.y) + out0 + c0 * p.ldy, p.ldy, cols, feats, lane);
        } else {
          store_32x32(buf16, v, p.bf16, static_cast<uint16_t*>(p.y) + out0 + c0 * p.ldy, p.ldy, cols, feats, lane);
        }
      };
      if (T.steps > kLongSteps) {
        // summed over the pieces in local memory (a piece's products take ten times as long), in loops of its own: the other
        // tiles keep their registers (one loop for both: weight gradient of short samples 81 -> 90 us)
        float sums[4][2][16];
        bool ok = true;
        for (int ks = 0; ok && ks < T.steps; ks += kLongSteps, ++count) {
          const int buf = count & 1;
          if (!(ok = wait_bar_warp(&S.acc_full[buf], (count >> 1) & 1, &S.waits))) break;
          fence_after();
#pragma unroll 1
          for (int c0 = c_first; c0 < T.cols; c0 += 64) {
            float v[2][16], (&sum)[2][16] = sums[c0 >> 6];
            ld_frags(tmem + buf * kAccCols + c0 + (static_cast<uint32_t>(32 * q) << 16), v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              sum[0][i] = ks ? sum[0][i] + v[0][i] : v[0][i];
              sum[1][i] = ks ? sum[1][i] + v[1][i] : v[1][i];
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster(lead_empty + 8 * buf);
        }
        if (!ok) break;
#pragma unroll 1
        for (int c0 = c_first; c0 < T.cols && feats > 0; c0 += 64) {
          float v[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = sums[c0 >> 6][0][i], v[1][i] = sums[c0 >> 6][1][i];
          if constexpr (kEpi == GM_ADAPT)
            if (S.ad.broken[n_tile & 15]) add_broken(v, p, T.c0 + c0, T.cols - c0, f0, lane);
          store(v, c0);
        }
        continue;
      }
      const int buf = count & 1;
      if (T.steps && !wait_bar_warp(&S.acc_full[buf], (count >> 1) & 1, &S.waits)) break;
      fence_after();
      // the accumulator goes back as soon as this warp has read its last columns, before they are stored
      const auto release = [&](int c0) {
        if (!T.steps || c0 + 64 < T.cols) return;
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lead_empty + 8 * buf);
      };
      if (c_first >= T.cols) release(c_first);
      for (int c0 = c_first; c0 < T.cols; c0 += 64) {
        float v[2][16];
        if (T.steps) {
          ld_frags(tmem + buf * kAccCols + c0 + (static_cast<uint32_t>(32 * q) << 16), v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = 0.f;
        }
        if constexpr (kEpi == GM_ADAPT)
          if (S.ad.broken[n_tile & 15] && feats > 0) add_broken(v, p, T.c0 + c0, T.cols - c0, f0, lane);
        release(c0);
        if (feats > 0) store(v, c0);
      }
      if (T.steps) ++count;
    }
    if (lead) store_wait<0>();   // the last stores have read this CTA's shared memory
  } else if (kEpi == GM_ADAPT && warp == 2 + kEpiWarps + kUWarps) {
    if constexpr (kEpi == GM_ADAPT) {
      // lists the distinct adapters of the tiles, ahead of the other roles
      uint32_t n_tile = 0;
      int e = 0;
      Tile T;
      for (; next_tile<kTake, true>(S, walk, lead_take, no_ask) && tile_at<kMode, kFeat>(S, p, walk.t, e, T); ++n_tile) {
        const int lb = n_tile % kLists;
        if (!wait_bar_warp(&S.ad.list_empty[lb], ((n_tile / kLists) & 1) ^ 1, &S.waits)) break;
        int id[8];
        uint32_t open[8];   // columns whose adapter is not listed yet, 32 at a time
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = 32 * i + lane;
          id[i] = c < T.cols ? p.ids[T.c0 + c] : -1;
          if (id[i] >= p.n_adapters || id[i] < 0) id[i] = -1;
          S.ad.id[lb][c] = id[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) open[i] = __ballot_sync(0xFFFFFFFFu, id[i] >= 0);
        int n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          while (open[i]) {
            const int a = __shfl_sync(0xFFFFFFFFu, id[i], __ffs(open[i]) - 1);
#pragma unroll
            for (int k = i; k < 8; ++k) open[k] &= ~__ballot_sync(0xFFFFFFFFu, id[k] == a);
            if (lane == 0) S.ad.list[lb][n] = a;
            ++n;
          }
        if (lane == 0) {
          S.ad.n_list[lb] = n;
          S.ad.broken[n_tile & 15] = 0;
        }
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&S.ad.list_full[lb]);
      }
    }
  } else if constexpr (kEpi == GM_ADAPT) {
    const int i0 = tid - 32 * (2 + kEpiWarps);
    const uint32_t lead_u = map_rank(smem_u32(S.ad.u_full), 0);
    uint32_t it = 0, tails = 0, n_tile = 0;
    bool alive = true;
    int e = 0;
    Tile T;
    pdl_wait();   // the u rows
    for (; next_tile<kTake, true>(S, walk, lead_take, no_ask) && tile_at<kMode, kFeat>(S, p, walk.t, e, T); ++n_tile) {
      const int lb = n_tile % kLists;
      if (!wait_bar_warp(&S.ad.list_full[lb], (n_tile / kLists) & 1, &S.waits)) break;
      const int n = S.ad.n_list[lb], blocks = (p.rank + 63) / 64, pairs = n * blocks;
      const int half = T.n / 2, c = rank * half + i0;   // this thread's column, one of this CTA's half
      const int mine = i0 < half ? S.ad.id[lb][c] : -1;
      int at0 = 0;
      for (int block = 0; block < blocks; ++block) {
        uint4 hi[8], lo[8];
        float odd = 0.f;
        const float* src = p.u + static_cast<size_t>(T.c0 + c) * p.rank + 64 * block;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const bool in = mine >= 0 && 64 * block + 8 * w < p.rank;
          // a sector of 32 bytes a load: as two of 16 it was fetched twice (70,000 rows 1,020 us against 970)
          uint64_t v[4] = {0, 0, 0, 0};
          if (in) load_u8(v, src + 8 * w);
          split_u(v, hi[w], lo[w], odd);
        }
        if (odd != 0.f)   // NaN
#pragma unroll
          for (int w = 0; w < 8; ++w)
            lo[w] = make_uint4(drop_odd(hi[w].x, lo[w].x), drop_odd(hi[w].y, lo[w].y), drop_odd(hi[w].z, lo[w].z),
                               drop_odd(hi[w].w, lo[w].w));
        for (int j = 0; j < n; ++j) {
          const int at = pair_at(block * n + j, pairs, T.steps);   // base steps before this pair
          it += at - at0;
          at0 = at;
          const bool use = mine == S.ad.list[lb][j];
          const int s = it % kStages, s2 = (it + 1) % kStages;
          it += 2;
          // B has landed and both stages are free (their own barriers' phases would be ambiguous here: these warps do
          // not see the steps in between)
          alive = alive && wait_bar_warp(&S.tail[s], (tails >> s) & 1, &S.waits);
          tails ^= 1u << s;
          if (i0 < half) {
            uint8_t *row = S.stage[s] + kHalf + 128 * i0, *row2 = S.stage[s2] + kHalf + 128 * i0;
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              *reinterpret_cast<uint4*>(row + 16 * (w ^ (i0 & 7))) = use ? hi[w] : zero;
              *reinterpret_cast<uint4*>(row2 + 16 * (w ^ (i0 & 7))) = use ? lo[w] : zero;
            }
          }
          uint4* words = reinterpret_cast<uint4*>(S.stage[s]) + i0;
          uint32_t any = 0;
          if (p.bf16) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const uint4 v = words[128 * w];
              const uint32_t bad = not_finite(v.x, 1) | not_finite(v.y, 1) | not_finite(v.z, 1) | not_finite(v.w, 1);
              if (bad) words[128 * w] = make_uint4(0, 0, 0, 0);
              any |= bad;
            }
          } else {
            uint4* words2 = reinterpret_cast<uint4*>(S.stage[s2]) + i0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              uint4 b_hi, b_lo;
              if (!split_f16(words[128 * w], b_hi, b_lo)) {
                b_hi = b_lo = make_uint4(0, 0, 0, 0);
                any = 1;
              }
              words[128 * w] = b_hi;
              words2[128 * w] = b_lo;
            }
          }
          if (any) S.ad.broken[n_tile & 15] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_cluster(lead_u + 8 * s);
        }
      }
      it += T.steps - at0;
      __syncwarp();
      if (lane == 0) mbarrier_arrive(&S.ad.list_empty[lb]);
    }
  } else if constexpr (kMode == GM_WGRAD) {
    // rows behind the group's end in its last stage belong to another expert (or to nobody, and may hold
    // anything): cleared in both operands, up to the end of the last k16 step that is issued
    const uint32_t lead_full = map_rank(smem_u32(S.full), 0);
    uint32_t it = 0, phases = 0;
    int e = 0;
    Tile T;
    while (next_tile<kTake, true>(S, walk, lead_take, no_ask) && tile_at<kMode, kFeat>(S, p, walk.t, e, T)) {
      it += T.steps;
      if (!(T.rows & 15)) continue;
      const int s = (it - 1) % kStages, lo = ((T.rows - 1) & 63) + 1, hi = (lo + 15) & ~15;
      if (!wait_bar_warp(&S.tail[s], (phases >> s) & 1, &S.waits)) break;
      phases ^= 1u << s;
      for (int i = lane; i < (hi - lo) * 32; i += 32) {   // four blocks of 64 x 128 bytes, eight 16-byte words a row
        const int blk = (i & 31) >> 3, word = i & 7, row = lo + (i >> 5);
        *reinterpret_cast<uint4*>(S.stage[s] + 8192 * blk + 128 * row + 16 * word) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_cluster(lead_full + 8 * s);
    }
  }
  fence_before();
  __syncthreads();
  if (S.waits.abort == 1) report_and_settle();
  cluster_sync();   // no CTA leaves while the other may still arrive on its barriers or read its stages
  fence_after();
  if (warp == 1) tmem_free<true>(tmem, 2 * kAccCols);
}

// ------------------------------------------------------------------ few rows per expert

constexpr int kSmallCols = 64;                   // most columns of a tile
constexpr int kSmallRing = 73728;                // 3 CTAs per SM: 4 stages of 16 columns, 3 of 64
constexpr int kMaxSplit = 8;                     // CTAs that share a tile's reduction
constexpr int kSmallPitch = 132;                 // floats between reduced columns
static_assert(kSmallCols * kSmallPitch * 4 <= kSmallRing, "the reduction reuses the ring");

// (B[id] u)[row][f .. f + 4) in fp32; 0 for a row without an adapter.
__device__ __forceinline__ float4 adapter_values(const GmParams& p, int row, int f) {
  const int id = p.ids[row];
  uint64_t d[4] = {0, 0, 0, 0};
  if (id >= 0 && id < p.n_adapters) {
    const uint16_t* b = p.b + (static_cast<size_t>(id) * p.feat + f) * p.rank;
    const float* u = p.u + static_cast<size_t>(row) * p.rank;
#pragma unroll 2
    for (int j = 0; j < p.rank; j += 8) {
      uint64_t uw[4], bw[4];
      load_u8(uw, u + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        widen8(bw, __ldg(reinterpret_cast<const uint4*>(b + static_cast<size_t>(i) * p.rank + j)), p.bf16);
#pragma unroll
        for (int w = 0; w < 4; ++w) fma_f32x2(d[i], bw[w], uw[w]);
      }
    }
  }
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s[i] = __uint_as_float(static_cast<uint32_t>(d[i])) + __uint_as_float(static_cast<uint32_t>(d[i] >> 32));
  return make_float4(s[0], s[1], s[2], s[3]);
}

// Four consecutive values of an output row.
__device__ __forceinline__ void store_out4(void* y, long long i, float4 v, int f32, int bf16) {
  if (f32)
    *reinterpret_cast<float4*>(static_cast<float*>(y) + i) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) = make_uint2(pack16(v.x, v.y, bf16), pack16(v.z, v.w, bf16));
}

template <int kMode, int kEpi>
__global__ void __launch_bounds__(192)
    k_grouped_small(const __grid_constant__ GmMaps maps, GmParams p, int split) {
  constexpr bool kTa = kMode == GM_DGRAD;
  constexpr int kFeat = kEpi == GM_GATED ? 64 : 128;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[8], empty[8], acc_full[2], acc_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ Waits s_waits;
  __shared__ int s_tile[4];   // expert, first row, rows
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), f0 = blockIdx.x / split * kFeat;

  if (warp == 1) {
    tmem_alloc<false>(&s_tmem, 2 * kSmallCols);
  } else if (tid == 64) {
    prefetch_map(&maps.a);
    s_waits.abort = 0;
    s_waits.limit = p.limit;
    for (int i = 0; i < 8; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    fence_mbar_init();
  }
  if (kEpi != GM_ADAPT) pdl_wait();   // adapters: nothing but the u rows comes from the previous kernel
  pdl_trigger();
  if (warp == 0) {
    // column tile blockIdx.y: an expert's rows in equal parts of at most kSmallCols.  A lane takes four experts at
    // a time, so that up to 128 experts' offsets are one round of loads.
    int base = 0;
    if (lane == 0) s_tile[2] = 0;
    __syncwarp();
    for (int e0 = 0; e0 < p.E; e0 += 128) {
      int off[5], c = 0;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int e = min(e0 + 4 * lane + i, p.E);
        off[i] = p.offsets ? clamp_off(p.offsets[e], p.m) : e * p.m;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) c += (max(off[i + 1] - off[i], 0) + kSmallCols - 1) / kSmallCols;
      int before = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
        if (lane >= d) before += o;
      }
      int at = static_cast<int>(blockIdx.y) - (base + before - c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rows = max(off[i + 1] - off[i], 0), nt = (rows + kSmallCols - 1) / kSmallCols;
        if (at >= 0 && at < nt) {
          const int width = ((rows + nt - 1) / nt + 15) & ~15;
          s_tile[0] = e0 + 4 * lane + i;
          s_tile[1] = off[i] + at * width;
          s_tile[2] = min(width, rows - at * width);
        }
        at -= nt;
      }
      base += __shfl_sync(0xFFFFFFFFu, before, 31);
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  const int expert = s_tile[0], row0 = s_tile[1], rows = s_tile[2];
  if (rows <= 0) {   // no such tile: the same for every CTA of the cluster
    if (warp == 1) tmem_free<false>(tmem, 2 * kSmallCols);
    return;
  }
  const int n = (rows + 15) & ~15;
  const int bytes = kHalf + n * 128, stages = min(8, kSmallRing / bytes);
  const int all = (p.red + 63) / 64, k0 = all * rank / split, steps = all * (rank + 1) / split - k0;
  const int seg = p.out_f32 ? kSegSteps : kLongSteps;   // pieces of the reduction, in two accumulators in turn

  if (warp == 0) {
    if (elect_one()) {
      for (int ks = 0; ks < min(steps, p.stall); ++ks) {
        const int s = ks % stages;
        if (!wait_bar(&empty[s], ((ks / stages) & 1) ^ 1, &s_waits)) break;
        const uint32_t a = smem_u32(ring) + s * bytes, bar = smem_u32(&full[s]);
        mbar_arrive_expect_tx(&full[s], bytes);
        const int k = 64 * (k0 + ks);
        if (kEpi == GM_GATED) {
          load_5d<false>(a, &maps.a, k, 0, 0, f0 / 16, expert, bar);
        } else if (kMode == GM_FWD) {
          load_3d<false>(a, &maps.a, k, f0, expert, bar);
        } else {
          load_3d<false>(a, &maps.a, f0, k, expert, bar);
          load_3d<false>(a + 8192, &maps.a, f0 + 64, k, expert, bar);
        }
        load_2d<false>(a + kHalf, &maps.b[n / 16 - 1], k, row0, bar);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = instr_desc(p.bf16, 128, n, kTa, false);
      bool go = true;
      for (int ks = 0, piece = 0; go && ks < steps; ++piece) {
        const int buf = piece & 1, end = min(ks + seg, steps);
        go = wait_bar(&acc_empty[buf], ((piece >> 1) & 1) ^ 1, &s_waits);
        fence_after();
        for (bool first = true; go && ks < end; ++ks) {
          const int s = ks % stages;
          if (!(go = wait_bar(&full[s], (ks / stages) & 1, &s_waits))) break;
          fence_after();
          const uint32_t a = smem_u32(ring) + s * bytes;
          const uint64_t da = tile_desc<kTa>(a), db = tile_desc<false>(a + kHalf);
          const int nk = (min(64, p.red - 64 * (k0 + ks)) + 15) / 16;
          for (int kk = 0; kk < nk; ++kk, first = false)
            mma<false>(tmem + buf * kSmallCols, da + kk * kStep16<kTa>, db + kk * kStep16<false>, idesc, !first);
          commit(&empty[s]);
        }
        if (go) commit(&acc_full[buf]);
      }
    }
  }
  __syncwarp();
  float* part = reinterpret_cast<float*>(ring);   // [column][kSmallPitch], after every product has read the ring
  // Columns rank, rank + split, ... of the tile are this CTA's to finish, one warp (GM_GATED: half a warp) a column
  // and four features a lane.
  constexpr int kLanes = kFeat / 4;
  const int i0 = tid - 64, fi = 4 * (i0 % kLanes), f = f0 + fi, first = rank + split * (i0 / kLanes);
  const int step = split * (128 / kLanes);
  constexpr int kEarly = kEpi == GM_ADAPT ? kSmallCols / kMaxSplit / 4 : 1;
  float4 delta[kEarly];
  bool ok = true;
  if (warp >= 2) {
    if (kEpi == GM_ADAPT && f < p.feat) {
      // the adapters' rows come to L2 before the weights queue up in front of them; B u while the weights stream, for
      // the first columns
      for (int c = first; c < rows; c += step) {
        const int id = p.ids[row0 + c];
        if (id >= 0 && id < p.n_adapters)
          for (int j = 0; j < 4 * p.rank; j += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.b + (static_cast<size_t>(id) * p.feat + f) * p.rank + j));
      }
      pdl_wait();
#pragma unroll
      for (int i = 0; i < kEarly; ++i)
        if (first + i * step < rows) delta[i] = adapter_values(p, row0 + first + i * step, f);
    }
    const int q = warp & 3;
    float acc[kSmallCols / 16][16];
#pragma unroll
    for (int j = 0; j < kSmallCols / 16; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
    for (int ks = 0, piece = 0; ok && ks < steps; ks += seg, ++piece) {
      const int buf = piece & 1;
      if (!(ok = wait_bar_warp(&acc_full[buf], (piece >> 1) & 1, &s_waits))) break;
      fence_after();
#pragma unroll
      for (int j = 0; j < kSmallCols / 16; ++j)
        if (16 * j < n) {
          float v[16];
          ld_cols16(tmem + buf * kSmallCols + 16 * j + (static_cast<uint32_t>(32 * q) << 16), v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j][i] += v[i];
        }
      fence_before();
      __syncwarp();
      if (lane == 0) mbarrier_arrive(&acc_empty[buf]);
    }
    if (ok)
#pragma unroll
      for (int j = 0; j < kSmallCols / 16; ++j)
        if (16 * j < n)
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(16 * j + i) * kSmallPitch + 32 * q + lane] = acc[j][i];
  }
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp >= 2 && ok) {
    const int lane_of = kEpi == GM_GATED ? (fi >> 4) * 32 + (fi & 15) : fi;
    uint32_t from[kMaxSplit];   // these features' first column in each CTA's part
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r) from[r] = map_rank(smem_u32(part) + lane_of * 4, min(r, split - 1));
    const auto add = [](float4& x, const float4& y) { x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w; };
    const auto finish = [&](int c, const float4& term) {
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      float4 pv[kMaxSplit], pu[kMaxSplit], v = zero, up = zero;
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r) {   // every load before the first sum; the sum in rank order
        pv[r] = ld_cluster_f32x4(from[r] + c * kSmallPitch * 4, r < split);
        if (kEpi == GM_GATED) pu[r] = ld_cluster_f32x4(from[r] + c * kSmallPitch * 4 + 64, r < split);
      }
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r) {
        add(v, pv[r]);
        if (kEpi == GM_GATED) add(up, pu[r]);
      }
      const long long row = row0 + c;
      if (kEpi == GM_GATED) {
        if (p.h) {
          store_out4(p.h, row * p.ldh + f, v, 0, p.bf16);
          store_out4(p.h, row * p.ldh + p.feat + f, up, 0, p.bf16);
        }
        v = make_float4(gelu16(v.x, p.gelu) * up.x, gelu16(v.y, p.gelu) * up.y, gelu16(v.z, p.gelu) * up.z,
                        gelu16(v.w, p.gelu) * up.w);
      }
      if (kEpi == GM_ADAPT) add(v, term);
      store_out4(p.y, row * p.ldy + f, v, p.out_f32, p.bf16);
    };
    int c = first;
    if (f < p.feat) {
      if (kEpi == GM_ADAPT) {
#pragma unroll
        for (int i = 0; i < kEarly; ++i, c += step)
          if (c < rows) finish(c, delta[i]);
      }
      for (; c < rows; c += step)
        finish(c, kEpi == GM_ADAPT ? adapter_values(p, row0 + c, f) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  if (s_waits.abort) report_and_settle();
  if (split > 1)
    cluster_sync();   // the others may still read this CTA's part
  else
    __syncthreads();
  if (warp == 1) tmem_free<false>(tmem, 2 * kSmallCols);
}

// ------------------------------------------------------------------ adapters' down half for many rows

// u[t] = scale[i] A[i] x[t] for 64 rows of x a cluster.  The distinct adapters
// of the rows go 128 / slot at a time (slot: the rank rounded up to a power of
// two) as the MMA's 128 features, for all 64 rows; a row keeps its own
// adapter's part.  The reduction is split over the cluster as above.
constexpr int kDownCols = 64;
constexpr int kDownStage = kHalf + kDownCols * 128;
constexpr int kDownStages = 4;
static_assert(kDownCols * kSmallPitch * 4 <= kDownStages * kDownStage, "the reduction reuses the ring");

__global__ void __launch_bounds__(192)
    k_adapter_down_many(const __grid_constant__ GmMaps maps, GmParams p, const float* scale, float* u, int slot, int split) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kDownStages], empty[kDownStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ Waits s_waits;
  __shared__ int s_n, s_list[64], s_nth[64];   // distinct adapters; which of them a row has, or -1
  uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), row0 = blockIdx.x / split * kDownCols,
            rows = min(kDownCols, p.m - row0);
  if (warp == 1) {
    tmem_alloc<false>(&s_tmem, 2 * kDownCols);
  } else if (tid == 64) {
    prefetch_map(&maps.a);
    prefetch_map(&maps.b[0]);
    s_waits.abort = 0;
    s_waits.limit = p.limit;
    for (int i = 0; i < kDownStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    int id[2], nth[2] = {-1, -1}, n = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      id[i] = lane + 32 * i < rows ? p.ids[row0 + lane + 32 * i] : -1;
      if (id[i] < 0 || id[i] >= p.n_adapters) id[i] = -1;
    }
    for (;;) {
      const uint32_t open0 = __ballot_sync(0xFFFFFFFFu, id[0] >= 0 && nth[0] < 0);
      const uint32_t open1 = __ballot_sync(0xFFFFFFFFu, id[1] >= 0 && nth[1] < 0);
      if (!(open0 | open1)) break;
      const int a = open0 ? __shfl_sync(0xFFFFFFFFu, id[0], __ffs(open0) - 1)
                          : __shfl_sync(0xFFFFFFFFu, id[1], __ffs(open1) - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (id[i] == a) nth[i] = n;
      if (lane == 0) s_list[n] = a;
      ++n;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) s_nth[lane + 32 * i] = nth[i];
    if (lane == 0) s_n = n;
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  const int n = s_n, each = 128 / slot;   // adapters of a pass
  const int all = (p.red + 63) / 64, k0 = all * rank / split, steps = all * (rank + 1) / split - k0;
  float* part = reinterpret_cast<float*>(ring);
  uint32_t from[kMaxSplit];
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r) from[r] = map_rank(smem_u32(part) + 16 * lane, min(r, split - 1));
  uint32_t it = 0, piece = 0;   // pieces of the reductions, in two accumulators in turn
  for (int a0 = each * blockIdx.y; a0 < n; a0 += each * gridDim.y) {
    const int na = min(each, n - a0);
    const uint32_t bytes = na * slot * 128 + kDownCols * 128;
    // after a wait that ran out the passes that are left are only met
    if (warp == 0) {
      if (elect_one() && !s_waits.abort) {
        for (int ks = 0; ks < steps && it + ks < static_cast<uint32_t>(p.stall); ++ks) {
          const uint32_t i = it + ks, s = i % kDownStages;
          if (!wait_bar(&empty[s], ((i / kDownStages) & 1) ^ 1, &s_waits)) break;
          const uint32_t a = smem_u32(ring) + s * kDownStage, bar = smem_u32(&full[s]);
          mbar_arrive_expect_tx(&full[s], bytes);
          for (int j = 0; j < na; ++j) load_3d<false>(a + j * slot * 128, &maps.a, 64 * (k0 + ks), 0, s_list[a0 + j], bar);
          load_2d<false>(a + kHalf, &maps.b[0], 64 * (k0 + ks), row0, bar);
        }
      }
    } else if (warp == 1) {
      if (elect_one() && !s_waits.abort) {
        const uint32_t idesc = instr_desc(p.bf16, 128, kDownCols, false, false);
        for (int ks = 0; ks < steps; ++ks) {
          const uint32_t i = it + ks, s = i % kDownStages, at = piece + ks / kLongSteps, buf = at & 1;
          if (ks % kLongSteps == 0 && !wait_bar(&acc_empty[buf], ((at >> 1) & 1) ^ 1, &s_waits)) break;
          if (!wait_bar(&full[s], (i / kDownStages) & 1, &s_waits)) break;
          fence_after();
          const uint32_t a = smem_u32(ring) + s * kDownStage;
          const uint64_t da = tile_desc<false>(a), db = tile_desc<false>(a + kHalf);
          const int nk = (min(64, p.red - 64 * (k0 + ks)) + 15) / 16;
          for (int kk = 0; kk < nk; ++kk)
            mma<false>(tmem + buf * kDownCols, da + kk * kStep16<false>, db + kk * kStep16<false>, idesc,
                       (ks % kLongSteps | kk) != 0);
          commit(&empty[s]);
          if ((ks + 1) % kLongSteps == 0 || ks + 1 == steps) commit(&acc_full[buf]);
        }
      }
    }
    __syncwarp();
    it += steps;
    bool ok = true;
    if (warp >= 2) {
      ok = __all_sync(0xFFFFFFFFu, !s_waits.abort);
      const int q = warp & 3;
      float acc[kDownCols / 16][16];
#pragma unroll
      for (int j = 0; j < kDownCols / 16; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
      for (int ks = 0, at = piece; ok && ks < steps; ks += kLongSteps, ++at) {
        const int buf = at & 1;
        if (!(ok = wait_bar_warp(&acc_full[buf], (at >> 1) & 1, &s_waits))) break;
        fence_after();
#pragma unroll
        for (int j = 0; j < kDownCols / 16; ++j) {
          float v[16];
          ld_cols16(tmem + buf * kDownCols + 16 * j + (static_cast<uint32_t>(32 * q) << 16), v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j][i] += v[i];
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&acc_empty[buf]);
      }
      if (ok)
#pragma unroll
        for (int j = 0; j < kDownCols / 16; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(16 * j + i) * kSmallPitch + 32 * q + lane] = acc[j][i];
    }
    piece += (steps + kLongSteps - 1) / kLongSteps;
    cluster_sync();
    fence_after();
    if (warp >= 2 && ok)
      for (int c = rank + split * (warp - 2); c < rows; c += 4 * split) {
        const int nth = s_nth[c], r = 4 * lane - (nth - a0) * slot;   // this lane's four ranks of the row's adapter
        if (nth < a0 || nth >= a0 + na || r < 0 || r >= min(slot, p.rank)) continue;
        const float sc = scale[s_list[nth]];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), pv[kMaxSplit];
#pragma unroll
        for (int j = 0; j < kMaxSplit; ++j) pv[j] = ld_cluster_f32x4(from[j] + c * kSmallPitch * 4, j < split);
#pragma unroll
        for (int j = 0; j < kMaxSplit; ++j) v.x += pv[j].x, v.y += pv[j].y, v.z += pv[j].z, v.w += pv[j].w;
        v.x *= sc, v.y *= sc, v.z *= sc, v.w *= sc;
        *reinterpret_cast<float4*>(u + static_cast<size_t>(row0 + c) * p.rank + r) = v;
      }
    fence_proxy_async_smem();   // the next pass's loads follow these accesses of the ring
    cluster_sync();             // the others may still read this CTA's part
  }
  __syncthreads();
  if (s_waits.abort) report_and_settle();
  if (warp == 1) tmem_free<false>(tmem, 2 * kDownCols);
}

// ------------------------------------------------------------------ launches

constexpr int kMaxKernels = 16;

// A wait's limit in 1024 cycles, and the loads after which a CTA's loading thread stops.
constexpr int kDefaultLimit = static_cast<int>(kSpinLimitCycles / 1024), kNever = std::numeric_limits<int>::max();
std::atomic<int> g_limit{kDefaultLimit}, g_stall{kNever};

GmParams with_limits(GmParams p) {
  p.limit = g_limit.load(std::memory_order_relaxed);
  p.stall = g_stall.load(std::memory_order_relaxed);
  return p;
}

struct DeviceInfo {
  int sms = 0;
};

bool device_info(DeviceInfo* d) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// rows [rows][cols] of 16-bit values, `ld` apart, in boxes of box_rows x 64
bool map_rows(CUtensorMap* m, const void* base, int cols, int rows, long long ld, int box_rows, bool bf16) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return encode_tiles(m, base, 2, dim, stride, box, bf16);
}

bool map_weights(CUtensorMap* m, const void* base, int E, int n, int k, int box_rows, bool bf16) {
  const cuuint64_t dim[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(k) * 2, static_cast<cuuint64_t>(k) * n * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return encode_tiles(m, base, 3, dim, stride, box, bf16);
}

// [E][2][f][k] seen as blocks of 16 features: a box is 64 k x 16 gate and the
// same 16 up rows of four blocks, so each warp's 32 accumulator lanes hold
// both halves of 16 features.
bool map_gated(CUtensorMap* m, const void* base, int E, int f, int k, bool bf16) {
  const cuuint64_t row = static_cast<cuuint64_t>(k) * 2;
  const cuuint64_t dim[5] = {static_cast<cuuint64_t>(k), 16, 2, static_cast<cuuint64_t>(f / 16),
                             static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[4] = {row, row * f, row * 16, row * 2 * f};
  const cuuint32_t box[5] = {64, 16, 2, 4, 1};
  return encode_tiles(m, base, 5, dim, stride, box, bf16);
}

// Dynamic shared memory past 48 KB has to be allowed once for a kernel and device.
template <typename K>
bool allow_smem(K kernel, size_t smem) {
  static std::atomic<uint64_t> done[kMaxKernels];   // devices, by kernel
  static std::atomic<const void*> known[kMaxKernels];
  int dev = 0, i = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const void* id = reinterpret_cast<const void*>(kernel);
  for (; i < kMaxKernels; ++i) {
    const void* at = known[i].load(std::memory_order_acquire);
    if (at == id || (!at && known[i].compare_exchange_strong(at, id)) || at == id) break;
  }
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (i < kMaxKernels && (done[i].load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  if (i < kMaxKernels) done[i].fetch_or(bit, std::memory_order_release);
  return true;
}

template <typename K>
bool launch(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, const GmMaps& maps,
            const GmParams& p, int split) {
  if (!allow_smem(kernel, smem)) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split ? 2 : 1;   // the persistent kernel's cluster is part of its type
  if constexpr (std::is_same_v<K, void (*)(GmMaps, GmParams)>)
    return cudaLaunchKernelEx(&cfg, kernel, maps, p) == cudaSuccess;
  else
    return cudaLaunchKernelEx(&cfg, kernel, maps, p, split) == cudaSuccess;
}

template <int kMode, int kEpi>
bool launch_big(const GmMaps& maps, const GmParams& p, int sms, cudaStream_t s) {
  constexpr int kFeat = kEpi == GM_GATED ? 128 : 256;
  const long long ft = (p.feat + kFeat - 1) / kFeat;
  const long long ct = kMode == GM_WGRAD ? static_cast<long long>(p.E) * ((p.cols + 255) / 256)
                                         : std::min(p.E, p.m) + static_cast<long long>(p.m) / 64;   // most parts, of 64
  const long long pairs = kTakes<kMode, kEpi> ? ft * ct : std::min<long long>(sms / 2, ft * ct);
  return launch(k_grouped<kMode, kEpi>, dim3(static_cast<unsigned>(2 * pairs)), BigCfg<kMode, kEpi>::kThreads,
                sizeof(BigSmem<kMode, kEpi>) + 1024, 2, s, maps, p, 0);
}

template <int kMode, int kEpi>
bool launch_small(const GmMaps& maps, const GmParams& p, int sms, cudaStream_t s) {
  constexpr int kFeat = kEpi == GM_GATED ? 64 : 128;
  const int ft = (p.feat + kFeat - 1) / kFeat, tiles = std::min(p.E, p.m) + p.m / kSmallCols;
  const int steps = (p.red + 63) / 64;
  // CTAs that share a tile's reduction: up to three on every SM (two with adapters, whose many columns make the sum over
  // the cluster dearer: 48 rows 17.7 us against 18.8), at least two k64 steps each, and eleven once every SM has one
  // (eight experts of 704 -> 2816, 176 tiles of 11 steps: 7.9 us whole against 8.8 halved; 32 of 512 -> 704 5.9 / 6.3; of
  // 22 steps 12.4 / 12.2).
  constexpr int kPerSm = kEpi == GM_ADAPT ? 2 : 3;
  const long long ctas = ft * static_cast<long long>(tiles);
  int split = 1;
  while (split < kMaxSplit && 2 * split * ctas <= kPerSm * sms && (split * ctas < sms ? 4 : 22) * split <= steps) split *= 2;
  return launch(k_grouped_small<kMode, kEpi>, dim3(ft * split, tiles), 192, kSmallRing + 1024, split, s, maps, p, split);
}

}  // namespace

void grouped_test_cycles(int64_t cycles) {
  g_limit = cycles > 0 ? static_cast<int>(std::min<int64_t>(cycles / 1024, kDefaultLimit)) : kDefaultLimit;
}

void grouped_test_loads(int64_t loads) { g_stall = loads > 0 && loads < kNever ? static_cast<int>(loads) : kNever; }

bool launch_adapter_down_many(const GmOperands& o, const GmParams& params, const float* scale, float* u, cudaStream_t s) {
  const GmParams p = with_limits(params);
  int slot = 8;
  while (slot < p.rank) slot *= 2;
  GmMaps maps;
  if (!map_weights(&maps.a, o.w, p.n_adapters, p.rank, o.k, slot, p.bf16) ||
      !map_rows(&maps.b[0], o.x, o.k, p.m, o.ldx, kDownCols, p.bf16))
    return false;
  const int blocks = (p.m + kDownCols - 1) / kDownCols, steps = (o.k + 63) / 64, most = std::min(kDownCols, p.n_adapters);
  DeviceInfo d;
  if (!device_info(&d)) return false;
  // one CTA an SM from the split, two with the shares of the adapters: measured 58 / 93 us (one adapter / runs of 41
  // rows, 4096 rows) against 62 / 97 with twice the split
  int split = 1;
  while (split < kMaxSplit && 2 * split * blocks <= d.sms && 4 * split <= steps) split *= 2;
  const int shares = std::max(1, std::min((most * slot + 127) / 128, 2 * d.sms / (split * blocks)));
  const size_t smem = kDownStages * kDownStage + 1024;
  if (!allow_smem(k_adapter_down_many, smem)) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(split * blocks, shares);   // x: more than 65535 blocks of rows are possible
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = split;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_adapter_down_many, maps, p, scale, u, slot, split) == cudaSuccess;
}

namespace {

// Few rows per expert: the small kernel.  Its tiles re-read an expert's weights (from L2) for every 64 rows, and its
// adapters cost a row's rank times the features on the ordinary pipes.  Small against persistent kernel, 128 experts:
// gated 2816 -> 704 at 4 rows an expert 125 us against 133, at 16 157 against 162, at 32 164 against 176; down 704 -> 2816
// 68 / 68, 83 / 82, 92 / 86.  Adapters at 2816 x 2816: 128 rows of rank 16 16 us against 24, of rank 64 30 against 26;
// 256 rows of rank 16 27 against 31.
bool few_rows(const GmParams& p) {
  if (p.offsets) return p.m <= 16 * static_cast<long long>(p.E);
  return p.m <= 64 || (p.m <= 256 && p.m * p.rank <= 4096);
}

}  // namespace

bool launch_grouped(int mode, int epi, const GmOperands& o, const GmParams& params, cudaStream_t s) {
  const GmParams p = with_limits(params);
  DeviceInfo d;
  if (!device_info(&d)) return false;
  GmMaps maps;
  if (mode == GM_WGRAD) {
    if (!map_rows(&maps.a, o.x, o.k, p.m, o.ldx, 64, p.bf16) || !map_rows(&maps.b[0], o.w, o.n, p.m, o.ldw, 64, p.bf16))
      return false;
    const cuuint64_t row = static_cast<cuuint64_t>(o.k) * 2;
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(o.k), static_cast<cuuint64_t>(o.n), static_cast<cuuint64_t>(p.E)};
    const cuuint64_t stride[2] = {row, row * o.n};
    if (!p.out_f32 && !encode_store(&maps.c, p.y, dim, stride, p.bf16)) return false;
    return p.out_f32 ? launch_big<GM_WGRAD, GM_F32>(maps, p, d.sms, s) : launch_big<GM_WGRAD, GM_PLAIN>(maps, p, d.sms, s);
  }
  const bool small = few_rows(p);
  // a tile has at most all of the rows, and at most kSmallCols or 256 (half of them a CTA)
  const int largest = small ? (std::min(p.m, kSmallCols) + 15) / 16 : ((std::min(p.m, 256) + 31) & ~31) / 32;
  for (int i = 0; i < largest; ++i)
    if (!map_rows(&maps.b[i], o.x, mode == GM_FWD ? o.k : o.n, p.m, o.ldx, 16 * (i + 1), p.bf16)) return false;
  if (epi == GM_GATED ? !map_gated(&maps.a, o.w, p.E, p.feat, o.k, p.bf16)
                      : !map_weights(&maps.a, o.w, p.E, o.n, o.k, mode == GM_FWD ? 128 : 64, p.bf16))
    return false;
  if (epi == GM_ADAPT && !small && !map_weights(&maps.c, p.b, p.n_adapters, p.feat, p.rank, 128, p.bf16)) return false;
  if (mode == GM_DGRAD)
    return small       ? launch_small<GM_DGRAD, GM_PLAIN>(maps, p, d.sms, s)
           : p.out_f32 ? launch_big<GM_DGRAD, GM_F32>(maps, p, d.sms, s)
                       : launch_big<GM_DGRAD, GM_PLAIN>(maps, p, d.sms, s);
  if (epi == GM_GATED)
    return small ? launch_small<GM_FWD, GM_GATED>(maps, p, d.sms, s) : launch_big<GM_FWD, GM_GATED>(maps, p, d.sms, s);
  if (epi == GM_ADAPT)
    return small ? launch_small<GM_FWD, GM_ADAPT>(maps, p, d.sms, s) : launch_big<GM_FWD, GM_ADAPT>(maps, p, d.sms, s);
  return small       ? launch_small<GM_FWD, GM_PLAIN>(maps, p, d.sms, s)
         : p.out_f32 ? launch_big<GM_FWD, GM_F32>(maps, p, d.sms, s)
                     : launch_big<GM_FWD, GM_PLAIN>(maps, p, d.sms, s);
}

bool grouped_gave_up(cudaStream_t s, bool* news) try {
  static std::mutex lock;
  static std::map<std::pair<int, cudaStream_t>, uint32_t> told;   // counts by device and stream
  int dev = 0;
  uint32_t count = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&count, g_gave_up, sizeof(count), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return false;
  {
    const std::lock_guard<std::mutex> hold(lock);
    const auto known = told.find({dev, s});
    *news = count != (known == told.end() ? 0u : known->second);
    if (*news) told[{dev, s}] = count;
  }
  if (!*news) return true;
  // the next replay of a graph that gave up does all of its work
  void* grid = nullptr;
  return cudaGetSymbolAddress(&grid, g_gave_up_grid) == cudaSuccess &&
         cudaMemsetAsync(grid, 0, sizeof(g_gave_up_grid), s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
} catch (...) {   // no memory for another stream's count
  return false;
}

}  // namespace moe
