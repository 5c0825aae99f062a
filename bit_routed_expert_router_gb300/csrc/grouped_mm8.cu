// Products of e4m3 rows grouped by expert with e4m3 weights on tcgen05, scales
// for blocks of 128 of the reduction on both sides:
//
//   y[r, n] = sum_b sx[r, b] sw[e][n / 128, b] sum_{k in b} x[r, k] w[e][n, k]
//
// and the gated form, whose output is e4m3 again with a scale for each 128 values.
//
// Persistent, one CTA an SM.  A tile is up to 128 rows of one expert
// by 256 weight rows: 256 features (128 where that makes few tiles), or gated the gate
// and the up rows of 128.  A
// block of 128 is one stage of 128-byte rows and four MMAs into one of two
// accumulators of 256 columns.  The MMA cannot scale by fp32 factors, so eight warps
// read every block's accumulator, multiply it by the factors and add it to sums in
// registers: 128 a thread, two at a time (fma.f32x2).  As the products of a block are
// exact and few, the sums are fp32's own.  The adding warps take registers from the
// others (setmaxnreg): 232 a thread.
//
// The rows are the MMA's M side, other than in the 16-bit products, although a ragged
// group then costs its rows rounded up to 128: a thread owns a row, so a block's factor
// is one value in a register (gated: two or three), and a row's 128 features that share
// a scale are two threads'.  With the features on the M side the factors change from
// column to column and came from shared memory, whose bandwidth the MMAs and the loads
// take: 1,600 cycles a block for what takes 340 alone, with CTA pairs 1,500 (shared
// expert's gate/up, 4096 rows: 144 and 90 us).
//
// What bounds it: few rows an expert, HBM (gated, 33 tokens of 128 experts, 2816 to
// 704 features: 67 us, 6.66 TB/s).  Many (shared expert's gate/up, 4096 rows, 2816 to
// 5632: 60 us, 2.17 PFLOP/s), the blocks: of 1,036 cycles an adding warp waits 220 for
// the accumulator, takes 107 for the factors, 443 to read and add, 146 for its share of
// a tile's end (3,200: stores) and 120 for the loop and what the two sides cost each
// other; alone the MMAs take 540, the reads 340, without the adding a block takes 907,
// without the loads 755.  Gated, 4096 tokens: 172 us, 1.51 PFLOP/s, in bursts; in a long
// row of calls 188 at the 1.78 GHz that the power cap leaves.  Pairs of CTAs on 256
// rows, which load a third less, take 58.9 us and, with ragged groups, 209.
#include <algorithm>
#include <cstddef>

#include "allow_smem.h"
#include "gelu16.cuh"
#include "grouped.h"
#include "moe.h"
#include "ops8.h"
#include "quant8.cuh"
#include "tensor_map.h"
#include "tile_regs.cuh"
#include "waits.cuh"

namespace moe {

namespace {

constexpr int kMaxE = 1024;
constexpr int kRows = 128;     // of a tile
constexpr int kMaxStages = 6, kRing = 196608;
constexpr int kAddWarps = 8, kThreads = 32 * (4 + kAddWarps);
constexpr int kRowMaps = 4;
constexpr int kOutBytes = 32 * 64;   // of an output buffer: 64 bytes of 32 rows, swizzled over their own width

struct Maps8 {
  CUtensorMap w;
  CUtensorMap x[kRowMaps];   // boxes of 16 << i rows
  CUtensorMap y;             // not gated: 64 bytes of 32 rows
};

struct Smem8 {
  uint8_t ring[kRing];
  float top[2][2][kRows];     // gated: rows' maxima over each half of the features, two tiles in turn
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], top_full, tile_full[4], tile_empty[4];
  uint32_t tmem;
  Waits waits;
  int4 tile[4];           // of the adding warps: expert, first feature, first row, rows; expert -1: no more
  int box;                // rows that a load takes at most: 16 << box
  // Behind it: the output's buffers (not gated: one or two for each adding warp), then the lists of the experts: their rows'
  // offsets, clamped to [0, m] and never going down, and the row tiles before each.
  alignas(1024) uint8_t rest[1];
};
constexpr int kMostSmem = 227 * 1024 - 1024;   // the struct starts at a multiple of 1024

// Bytes behind Smem8's fixed part; two buffers a warp where the lists leave room.
__host__ __device__ __forceinline__ int out_buffers(bool gated, int E) {
  const int fixed = static_cast<int>(offsetof(Smem8, rest)) + 8 * (E + 1);
  return gated ? 0 : fixed + 2 * kAddWarps * kOutBytes <= kMostSmem ? 2 : 1;
}
static_assert(offsetof(Smem8, rest) + kAddWarps * kOutBytes + 8 * (kMaxE + 1) <= kMostSmem, "one CTA per SM");

// The lists behind the buffers.
struct Lists {
  int *off, *tiles;
  __device__ __forceinline__ Lists(Smem8& S, bool gated, int E)
      : off(reinterpret_cast<int*>(S.rest + out_buffers(gated, E) * kAddWarps * kOutBytes)), tiles(off + E + 1) {}
};

struct Tile {
  int e, f0;      // expert, first feature
  int r0, rows;   // first row of x, rows
};

// Tile t in the order expert, feature tile, row tile; a whole warp, which looks at 32 experts at a time (one after the other they
// took longer than some tiles).  e: the last tile's expert.
__device__ __forceinline__ bool tile_at(const Lists& L, int E, int ft, int feats, int t, int& e, Tile& T) {
  const int lane = threadIdx.x & 31;
  uint32_t later = 0;
  for (; e < E; e += 32) {
    later = __ballot_sync(0xFFFFFFFFu, e + lane < E && L.tiles[min(e + lane, E - 1) + 1] * ft > t);
    if (later) break;
  }
  if (!later) return false;
  e += __ffs(later) - 1;
  const int nt = L.tiles[e + 1] - L.tiles[e], rem = t - L.tiles[e] * ft, f = rem / nt, c = rem - f * nt;
  const int lo = L.off[e];
  T.e = e;
  T.f0 = f * feats;
  T.r0 = lo + c * kRows;
  T.rows = min(kRows, L.off[e + 1] - T.r0);
  return true;
}

// The box of a load of `rows` rows.
__device__ __forceinline__ int box_of(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

// Offsets clamped and made to never go down, and the number of row tiles before each expert; one warp.
__device__ void list_tiles(Smem8& S, const Lists& L, const int32_t* offsets, int E, int m) {
  const int lane = threadIdx.x & 31;
  int base = 0, before = 0, most = 0;
  if (lane == 0) L.tiles[0] = 0;
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= E ? clamp_off(offsets[e], m) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, before);
    if (e <= E) L.off[e] = v;
    const int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1), rows = e > 0 && e <= E ? v - (lane ? prev : before) : 0;
    const int nt = (rows + kRows - 1) / kRows;
    most = max(most, min(rows, kRows));
    int c = nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, c, d);
      if (lane >= d) c += o;
    }
    if (e > 0 && e <= E) L.tiles[e] = base + c;
    base += __shfl_sync(0xFFFFFFFFu, c, 31);
    before = __shfl_sync(0xFFFFFFFFu, v, 31);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) S.box = box_of(most);
}

__device__ __forceinline__ void store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}

// kind::f8f6f4: fp32 accumulators, e4m3 operands, both K-major, M x N.
__host__ __device__ constexpr uint32_t instr_desc8(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

template <int kRegs>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
// 384 threads are launched with 168 registers each: 128 x 40 + 256 x 232 are the same 64,512.
constexpr int kFewRegs = 40, kManyRegs = 232;

// 16 columns of this thread's accumulator lane: issued, and waited for.  The wait takes the registers, so that nothing uses them
// before it.
struct Cols16 {
  uint32_t r[16];
  __device__ __forceinline__ void issue(uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
  }
  __device__ __forceinline__ void wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  }
  __device__ __forceinline__ uint64_t pair(int i) const { return static_cast<uint64_t>(r[2 * i + 1]) << 32 | r[2 * i]; }
};

// GELU(g) u of two features.  The tanh form: g / (1 + 2^z) u, z = -2 log2(e) sqrt(2 / pi) (g + 0.044715 g^3); past fp32's range
// 2^z is infinite and the quotient 0.
template <int kGelu>
__device__ __forceinline__ uint64_t gated_pair(uint64_t g, uint64_t u) {
  if constexpr (kGelu == MOE_GELU_TANH) {
    constexpr float c = -2.f * 1.4426950408889634f * 0.7978845608028654f;
    uint64_t s = pack_f32x2(c, c);
    fma_f32x2(s, mul_f32x2(g, g), pack_f32x2(0.044715f * c, 0.044715f * c));
    const uint64_t z = mul_f32x2(g, s);
    float e[2], r[2];
    asm("ex2.approx.f32 %0, %1;" : "=f"(e[0]) : "f"(lo_f32(z)));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e[1]) : "f"(hi_f32(z)));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r[0]) : "f"(1.f + e[0]));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r[1]) : "f"(1.f + e[1]));
    return mul_f32x2(mul_f32x2(g, pack_f32x2(r[0], r[1])), u);
  } else {
    return pack_f32x2(gelu16(lo_f32(g), kGelu) * lo_f32(u), gelu16(hi_f32(g), kGelu) * hi_f32(u));
  }
}

// The scales of a block that an adding thread needs: of its row, and of its columns' blocks of weight rows (gated: of the gate
// rows, of the up rows, and where these are rows of two blocks, of the second one).
template <bool kGated>
struct Scales {
  const float *sx, *sg, *su;
  int second;   // from su's row of scales to the second block's; 0: there is none
  float x, g, u, u2;
  __device__ __forceinline__ void load() {
    x = *sx++;
    g = __ldg(sg++);
    if (kGated) {
      if (second) u2 = __ldg(su + second);
      u = __ldg(su++);
    }
  }
};

// kGelu: -1 not gated, else the variant; kWeightRows: of a tile, 256 or (not gated) 128
template <int kGelu, int kWeightRows>
__global__ void __launch_bounds__(kThreads, 1) k_grouped8(const __grid_constant__ Maps8 maps, const __grid_constant__ Mm8Params p) {
  constexpr bool kGated = kGelu >= 0;
  constexpr int kFeats = kGated ? kWeightRows / 2 : kWeightRows;   // of a tile
  constexpr int kW = kWeightRows * 128;                            // bytes of its weights in a stage
  constexpr int kMine = kWeightRows / 2, kHalf = kFeats / 2;       // columns of a thread; features of a half of the warps
  extern __shared__ uint8_t smem_raw[];
  Smem8& S = *reinterpret_cast<Smem8*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Lists L(S, kGated, p.E);
  const int feats = kGated ? p.n / 2 : p.n, ft = (feats + kFeats - 1) / kFeats, blocks = (p.k + 127) / 128;

  if (tid == 0) {
    prefetch_map(&maps.w);
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.acc_full[i], 1);
      mbar_init(&S.acc_empty[i], kAddWarps);
    }
    mbar_init(&S.top_full, kAddWarps);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.tile_full[i], 1);
      mbar_init(&S.tile_empty[i], kAddWarps);
    }
    S.waits.abort = 0;
    S.waits.limit = p.limit;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<false>(&S.tmem, 2 * kWeightRows);
  pdl_wait();
  pdl_trigger();
  if (warp == 0) list_tiles(S, L, p.offsets, p.E, p.m);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S.tmem;
  // few rows leave room for more stages (the MMA reads 128 rows all the same: the ring goes on behind the last stage)
  const int stage_bytes = kW + (2048 << S.box), stages = min(kMaxStages, (kRing - (16384 - (2048 << S.box))) / stage_bytes);
  int e = 0;
  Tile T;

  if (warp < 4) {
    give_registers<kFewRegs>();
    if (warp == 0) {
      int it = 0, s = 0;
      uint32_t phase = 1;
      bool go = true;
      for (int t = blockIdx.x; go && tile_at(L, p.E, ft, kFeats, t, e, T); t += gridDim.x) {
        const int box = box_of(T.rows);
        if (elect_one())
          for (int b = 0; b < blocks; ++b) {
            if (!(go = it + b < p.stall && wait_bar(&S.empty[s], phase, &S.waits))) break;
            mbar_arrive_expect_tx(&S.full[s], kW + (2048 << box));
            const uint32_t w = smem_u32(S.ring) + s * stage_bytes, bar = smem_u32(&S.full[s]);
            load_3d<false>(w, &maps.w, 128 * b, T.f0, T.e, bar);
            if (kWeightRows > 128) load_3d<false>(w + kW / 2, &maps.w, 128 * b, kGated ? feats + T.f0 : T.f0 + 128, T.e, bar);
            load_2d<false>(w + kW, &maps.x[box], 128 * b, T.r0, bar);
            if (++s == stages) s = 0, phase ^= 1;
          }
        it += blocks;
        go = __all_sync(0xFFFFFFFFu, go);
      }
    } else if (warp == 1) {
      if (elect_one()) {
        constexpr uint32_t idesc = instr_desc8(kRows, kWeightRows);
        int it = 0, s = 0;
        uint32_t phase = 0;
        bool go = true;
        for (int t = blockIdx.x; go && t < L.tiles[p.E] * ft; t += gridDim.x) {
          for (int b = 0; b < blocks; ++b, ++it) {
            const int buf = it & 1;
            if (!(go = wait_bar(&S.full[s], phase, &S.waits) && wait_bar(&S.acc_empty[buf], ((it >> 1) & 1) ^ 1, &S.waits))) break;
            fence_after();
            const uint32_t w = smem_u32(S.ring) + s * stage_bytes;
            const uint64_t da = tile_desc<false>(w + kW), db = tile_desc<false>(w);
            const int steps = (min(128, p.k - 128 * b) + 31) / 32;
            for (int i = 0; i < steps; ++i) mma8(tmem + buf * kWeightRows, da + 2 * i, db + 2 * i, idesc, i != 0);
            commit(&S.acc_full[buf]);
            commit(&S.empty[s]);
            if (++s == stages) s = 0, phase ^= 1;
          }
        }
      }
    } else if (warp == 2) {
      bool go = true, more = true;
      for (int t = blockIdx.x, n = 0; go && more; t += gridDim.x, ++n) {   // the adding warps' tiles
        more = tile_at(L, p.E, ft, kFeats, t, e, T);
        if (!(go = wait_bar_warp(&S.tile_empty[n & 3], ((n >> 2) & 1) ^ 1, &S.waits))) break;
        if (lane == 0) {
          S.tile[n & 3] = make_int4(more ? T.e : -1, T.f0, T.r0, T.rows);
          mbarrier_arrive(&S.tile_full[n & 3]);
        }
      }
    }
  } else {
    take_registers<kManyRegs>();
    const int q = warp & 3, half = (warp - 4) >> 2;   // this warp's lanes of tensor memory, its half of the columns
    const int rows_w = (p.n + 127) / 128;             // blocks of weight rows
    const int r = 32 * q + lane;                      // this thread's row of a tile
    Scales<kGated> sc;
    sc.u2 = 0.f;
    const auto start = [&](const Tile& T) {
      const int f0 = T.f0 + kHalf * half;
      sc.sx = p.sx + static_cast<long long>(max(T.r0 + min(r, T.rows - 1), 0)) * blocks;
      const float* sw = p.sw + static_cast<long long>(T.e) * rows_w * blocks;
      sc.sg = sw + min(f0 / 128, rows_w - 1) * blocks;
      if constexpr (kGated) {
        const int up = feats + f0, block = min(up / 128, rows_w - 1);
        sc.su = sw + block * blocks;
        sc.second = up % 128 > 64 && block + 1 < rows_w ? blocks : 0;
      }
      sc.load();
    };
    [[maybe_unused]] const int n_buf = out_buffers(kGated, p.E);
    [[maybe_unused]] uint32_t n_part = 0;
    int it = 0, n_tile = 0;
    bool ok = true, more = false;
    const auto next_tile = [&](int n) {
      if (!(ok = wait_bar_warp(&S.tile_full[n & 3], (n >> 2) & 1, &S.waits))) return;
      const int4 v = S.tile[n & 3];
      __syncwarp();
      if (lane == 0) mbarrier_arrive(&S.tile_empty[n & 3]);
      T.e = v.x, T.f0 = v.y, T.r0 = v.z, T.rows = v.w;
      if ((more = v.x >= 0)) start(T);
    };
    next_tile(0);
    for (; ok && more; ++n_tile) {
      const bool rows_here = 32 * q < T.rows;
      // The sums of this thread's columns, two a register pair.  Plain: features f0 ..; gated: 64 gate columns, then their up columns.
      const int f0 = T.f0 + kHalf * half;
      uint64_t acc[kMine / 2];
#pragma unroll
      for (int j = 0; j < kMine / 2; ++j) acc[j] = 0;
      const int in_first = ((feats + f0) / 128 + 1) * 128 - (feats + f0);   // up rows in the first of their blocks
      const uint32_t at0 = tmem + (static_cast<uint32_t>(32 * q) << 16) + kHalf * half;
      for (int b = 0; b < blocks; ++b, ++it) {
        const int buf = it & 1;
        if (!(ok = wait_bar_warp(&S.acc_full[buf], (it >> 1) & 1, &S.waits))) break;
        fence_after();
        // this block's factors; the next one's scales are on their way while it is added
        const float f[3] = {sc.x * sc.g, kGated ? sc.x * sc.u : 0.f, kGated ? sc.x * sc.u2 : 0.f};
        if (b + 1 < blocks) sc.load();
        if (rows_here) {
          const uint32_t at = at0 + buf * kWeightRows;
          const auto column = [](int i) { return kGated ? 16 * (i & 3) + 128 * (i >> 2) : 16 * i; };
          Cols16 v[2];
          v[0].issue(at);
#pragma unroll
          for (int i = 0; i < kMine / 16; ++i) {
            v[i & 1].wait();
            if (i < kMine / 16 - 1) {
              v[(i + 1) & 1].issue(at + column(i + 1));
            } else {   // the accumulator is given back
              fence_before();
              __syncwarp();
              if (lane == 0) mbarrier_arrive(&S.acc_empty[buf]);
            }
            const float now = !kGated || i < 4 ? f[0] : 16 * (i & 3) < in_first ? f[1] : f[2];
            const uint64_t f2 = pack_f32x2(now, now);
#pragma unroll
            for (int j = 0; j < 8; ++j) fma_f32x2(acc[8 * i + j], v[i & 1].pair(j), f2);
          }
        } else {
          fence_before();
          __syncwarp();
          if (lane == 0) mbarrier_arrive(&S.acc_empty[buf]);
        }
      }
      if (!ok) break;
      const Tile D = T;   // done; the next tile's first scales come while it is stored
      next_tile(n_tile + 1);
      if (!ok) break;
      if constexpr (kGated) {
        // a in the gate values' place, and its largest magnitude
        float top = 0.f;
        if (rows_here)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (f0 + 16 * i >= feats) break;
#pragma unroll
            for (int j = 8 * i; j < 8 * i + 8; ++j) {
              acc[j] = gated_pair<kGelu>(acc[j], acc[32 + j]);
              top = max_abs(max_abs(top, lo_f32(acc[j])), hi_f32(acc[j]));
            }
          }
        S.top[n_tile & 1][half][r] = top;
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&S.top_full);
        if (!(ok = wait_bar_warp(&S.top_full, n_tile & 1, &S.waits))) break;
        // (two tiles' maxima in turn: who writes one again knows that all have come to the tile between)
        const Scale8 s8 = scale8(max_abs(top, S.top[n_tile & 1][half ^ 1][r]));
        if (r < D.rows) {
          const long long row = D.r0 + r;
          if (half == 0) p.sa[row * ((feats + 127) / 128) + D.f0 / 128] = s8.scale;
          uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + row * p.ldy + f0);
          const uint64_t x2 = pack_f32x2(s8.inverse, s8.inverse);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t a = mul_f32x2(acc[8 * i + 2 * j], x2), c = mul_f32x2(acc[8 * i + 2 * j + 1], x2);
              w[j] = to_e4m3x4(lo_f32(a), hi_f32(a), lo_f32(c), hi_f32(c));
            }
            if (f0 + 16 * i < feats) out[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else if (rows_here) {
        // 64 bytes of 32 rows at a time through the warp's own buffers: the TMA engine writes one out while the next is filled,
        // where all 32 rows are the tile's; of the last ones each row's words go out by themselves.  (Read back and stored by
        // the warps, 64 bytes of eight rows an instruction, all of them took 2,500 cycles a tile: down, 4096 tokens, 114 us.)
        const bool wide = p.out == MOE_F32, whole = 32 * q + 32 <= D.rows;
        const int n_parts = kMine / (wide ? 16 : 32), each = wide ? 16 : 32;   // features of a part
        // the first of this lane's rows and words where rows go out by themselves
        const int row0 = 32 * q + (lane >> 2), first = f0 + each / 4 * (lane & 3);
        uint8_t* const out = static_cast<uint8_t*>(p.y) + ((D.r0 + row0) * p.ldy + first) * (wide ? 4 : 2);
        const long long step = 8 * p.ldy * (wide ? 4 : 2);
#pragma unroll
        for (int i = 0; i < kMine / 16; ++i) {
          if (i >= n_parts || f0 + each * i >= feats) break;
          uint8_t* const buf = S.rest + ((n_buf == 2 ? n_part & 1 : 0) * kAddWarps + warp - 4) * kOutBytes;
          ++n_part;
          if (lane == 0) {   // (this lane issues all of the warp's stores)
            if (n_buf == 2 && whole)   // (parts that are not whole commit nothing that could be counted)
              store_wait<1>();
            else
              store_wait<0>();
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 w;
            if (wide) {
              const uint64_t a = acc[8 * i + 2 * j], c = acc[8 * i + 2 * j + 1];
              w = make_uint4(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(c),
                             static_cast<uint32_t>(c >> 32));
            } else {
              const uint64_t* a = acc + (16 * i + 4 * j) % (kMine / 2);
              const int bf16 = p.out == MOE_BF16;
              w = make_uint4(pack16(lo_f32(a[0]), hi_f32(a[0]), bf16), pack16(lo_f32(a[1]), hi_f32(a[1]), bf16),
                             pack16(lo_f32(a[2]), hi_f32(a[2]), bf16), pack16(lo_f32(a[3]), hi_f32(a[3]), bf16));
            }
            *reinterpret_cast<uint4*>(buf + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) = w;
          }
          if (whole) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) store_2d(&maps.y, smem_u32(buf), f0 + each * i, D.r0 + 32 * q);
            continue;
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (32 * q + 8 * j >= D.rows) break;
            if (row0 + 8 * j < D.rows && first + each * i < feats)
              *reinterpret_cast<uint4*>(out + j * step + 64 * i) =
                  *reinterpret_cast<const uint4*>(buf + 64 * (8 * j + (lane >> 2)) + 16 * ((lane & 3) ^ ((lane >> 3) & 3)));
          }
        }
      }
    }
    if (!kGated && lane == 0) store_wait<0>();   // before the buffers go
  }
  fence_before();
  __syncthreads();
  if (S.waits.abort == 1) report_and_settle(p.gave_up);
  fence_after();
  if (warp == 1) tmem_free<false>(tmem, 2 * kWeightRows);
}

// ------------------------------------------------------------------ launches

bool map_rows8(CUtensorMap* m, const void* base, int k, int rows, long long ld, int box_rows) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  return encode_byte_tiles(m, base, 2, dim, stride, box);
}

bool map_weights8(CUtensorMap* m, const void* base, int E, int n, int k) {
  const cuuint64_t dim[3] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(k) * n};
  const cuuint32_t box[3] = {128, 128, 1};
  return encode_byte_tiles(m, base, 3, dim, stride, box);
}

// Stores of 64 bytes of 32 rows, swizzled over their own width.
bool map_out(CUtensorMap* m, const Mm8Params& p) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const int size = p.out == MOE_F32 ? 4 : 2;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(p.n), static_cast<cuuint64_t>(p.m)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(p.ldy) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / size), 32}, ones[2] = {1, 1};
  return encode &&
         encode(m, p.out == MOE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                   : p.out == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                2, p.y, dim, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tiles at most, with `weight_rows` weight rows each.
long long most_tiles(const Mm8Params& p, int weight_rows) {
  return (p.n + weight_rows - 1) / weight_rows * (std::min(p.E, p.m) + static_cast<long long>(p.m) / kRows);
}

template <int kGelu, int kWeightRows>
bool launch(const Maps8& maps, const Mm8Params& p, int sms, cudaStream_t s) {
  const long long most = most_tiles(p, kWeightRows);
  const size_t smem = offsetof(Smem8, rest) + out_buffers(kGelu >= 0, p.E) * kAddWarps * kOutBytes + 8 * (p.E + 1) + 1024;
  if (!allow_smem(k_grouped8<kGelu, kWeightRows>, kMostSmem + 1024)) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(sms, most)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_grouped8<kGelu, kWeightRows>, maps, p) == cudaSuccess;
}

}  // namespace

bool launch_grouped8(bool gated, const Mm8Params& params, cudaStream_t s) {
  Mm8Params p = params;
  const WaitLimits l = wait_limits();
  p.limit = l.cycles1024, p.stall = l.loads;
  if (!(p.gave_up = gave_up_here())) return false;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  Maps8 maps;
  const int most = std::min(p.m, kRows);
  for (int i = 0; i < kRowMaps && (i == 0 || 8 << i < most); ++i)
    if (!map_rows8(&maps.x[i], p.x, p.k, p.m, p.ldx, 16 << i)) return false;
  if (!map_weights8(&maps.w, p.w, p.E, p.n, p.k)) return false;
  if (!gated && !map_out(&maps.y, p)) return false;
  // Tiles of half the weight rows where all of them start at once (one group of 1000 rows, 2816 to 512: 13.7 -> 11.0 us; 4 experts
  // of 4 rows, 2816 to 1408: 13.0 -> 10.0); where they do not, they cost (8 rows of as many experts, 704 to 2816: 8.3 -> 9.3).
  if (!gated) return most_tiles(p, 128) <= sms ? launch<-1, 128>(maps, p, sms, s) : launch<-1, 256>(maps, p, sms, s);
  return p.gelu == MOE_GELU_TANH ? launch<MOE_GELU_TANH, 256>(maps, p, sms, s) : launch<MOE_GELU_ERF, 256>(maps, p, sms, s);
}

}  // namespace moe
