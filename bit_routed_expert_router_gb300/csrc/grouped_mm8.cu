// Products of e4m3 rows grouped by expert with e4m3 weights on tcgen05, scales
// for blocks of 128 of the reduction on both sides:
//
//   y[r, n] = sum_b sx[r, b] sw[e][n / 128, b] sum_{k in b} x[r, k] w[e][n, k]
//
// and the gated form, whose output is e4m3 again with a scale for each 128 values.
//
// Persistent pairs of CTAs, as the 16-bit products: 256 weight rows on the MMA's M
// side (cta_group::2), up to 256 rows of x on its N side, an expert's rows cut into
// equal parts.  A block of 128 is one stage of 128-byte rows and four MMAs into one
// of two accumulators.  The MMA cannot scale by fp32 factors, so eight warps read
// every block's accumulator, multiply it by the factors and add it to sums in
// registers: 128 a thread, two at a time (fma.f32x2).  As the products of a block
// are exact and few, the sums are fp32's own.  Four warps turn the rows' scales,
// which lie row by row, into one array a block that the adding warps read as pairs;
// the weights' scale of a block is one value for a warp.  The adding warps take
// registers from the others (setmaxnreg): 208 a thread.
//
// Gated: 16 gate and the same 16 up rows in each warp's lanes, so that a thread ends
// with both factors; the 128 values that share a scale lie in both CTAs, which
// exchange their maxima through distributed shared memory.
#include <algorithm>
#include <limits>

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
constexpr int kStages = 5, kStageBytes = 32768, kHalf = 16384;   // 128 weight rows, and up to 128 rows of x
constexpr int kAccCols = 256;
constexpr int kAddWarps = 8, kScaleWarps = 4, kThreads = 32 * (4 + kAddWarps + kScaleWarps);
constexpr int kScaleBlocks = 4, kScaleStages = 4;                // blocks of a stage of the rows' scales
constexpr int kRowMaps = 8;

struct Maps8 {
  CUtensorMap a;
  CUtensorMap b[kRowMaps];   // boxes of 16 (i + 1) rows of x
};

struct Smem8 {
  uint8_t stage[kStages][kStageBytes];
  float sx[kScaleStages][kScaleBlocks][256];
  alignas(16) uint8_t epi[kAddWarps][4 * 8 * kEpiPitch];
  uint32_t top[2][2][4][256];   // gated: columns' maxima, two tiles in turn, of each CTA and quarter of its lanes
  float inverse[2][256];
  uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], sx_full[kScaleStages], sx_empty[kScaleStages], top_full, inverse_full;
  uint32_t tmem;
  Waits waits;
  int off[kMaxE + 1];     // clamped to [0, m], never going down
  int tiles[kMaxE + 1];   // column tiles before each expert
};
static_assert(sizeof(Smem8) + 1024 <= 227 * 1024, "one CTA per SM");

struct Tile {
  int e, f0;         // expert, first feature (gated: of a)
  int c0, cols, n;   // first row of x, rows, rows rounded up for the MMA
};

// Tile t in the order expert, feature tile, column tile.
template <int kFeat>
__device__ __forceinline__ bool tile_at(const Smem8& S, int E, int feats, int t, int& e, Tile& T) {
  const int ft = (feats + kFeat - 1) / kFeat;
  while (e < E && S.tiles[e + 1] * ft <= t) ++e;
  if (e >= E) return false;
  const int nt = S.tiles[e + 1] - S.tiles[e], rem = t - S.tiles[e] * ft, f = rem / nt, c = rem - f * nt;
  const int lo = S.off[e], rows = S.off[e + 1] - lo, width = ((rows + nt - 1) / nt + 31) & ~31;
  T.e = e;
  T.f0 = f * kFeat;
  T.c0 = lo + c * width;
  T.cols = min(width, lo + rows - T.c0);
  T.n = max((T.cols + 31) & ~31, 32);   // the last part of a group may be empty
  return true;
}

// Offsets clamped and made to never go down, and the number of column tiles before each expert; one warp.  Parts of at most 256
// rows; of 128 or 64 where the tiles then still are one round of the pairs.
template <int kFeat>
__device__ void list_tiles(Smem8& S, const int32_t* offsets, int E, int m, int feats) {
  const int lane = threadIdx.x & 31;
  int n128 = 0, n64 = 0;
  for (int e0 = 0, before = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= E ? clamp_off(offsets[e], m) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, before);
    if (e <= E) S.off[e] = v;
    const int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1), rows = v - (lane ? prev : before);
    if (e > 0 && e <= E) n128 += (rows + 127) / 128, n64 += (rows + 63) / 64;
    before = __shfl_sync(0xFFFFFFFFu, v, 31);
  }
  __syncwarp();
  n128 = __reduce_add_sync(0xFFFFFFFFu, n128);
  n64 = __reduce_add_sync(0xFFFFFFFFu, n64);
  const int ft = (feats + kFeat - 1) / kFeat, pairs = gridDim.x >> 1;
  const int width = n64 * ft <= pairs ? 64 : n128 * ft <= pairs ? 128 : 256;
  int base = 0;
  if (lane == 0) S.tiles[0] = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int c = e < E ? (S.off[e + 1] - S.off[e] + width - 1) / width : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, c, d);
      if (lane >= d) c += o;
    }
    if (e < E) S.tiles[e + 1] = base + c;
    base += __shfl_sync(0xFFFFFFFFu, c, 31);
  }
}

// kind::f8f6f4: fp32 accumulators, e4m3 operands, both K-major, M x N.
__host__ __device__ constexpr uint32_t instr_desc8(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
// 512 threads are launched with 128 registers each: 256 x 48 + 256 x 208 are the same 65,536.
constexpr int kFewRegs = 48, kManyRegs = 208;

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float lo_f32(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_f32(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

// A release to the pair, whose other CTA reads what this warp wrote to its shared memory.
__device__ __forceinline__ void arrive_release_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// The weights' scales of a warp's rows, 32 blocks at a time: lane i holds that of block i.
struct RowScales {
  const float* from;
  float mine;
  __device__ __forceinline__ float at(int b, int blocks, int lane) {
    if ((b & 31) == 0) mine = b + lane < blocks ? __ldg(from + b + lane) : 0.f;
    return __shfl_sync(0xFFFFFFFFu, mine, b & 31);
  }
};

template <bool kGated>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_grouped8(const __grid_constant__ Maps8 maps, const __grid_constant__ Mm8Params p) {
  constexpr int kFeat = kGated ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  Smem8& S = *reinterpret_cast<Smem8*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int feats = kGated ? p.n / 2 : p.n, blocks = (p.k + 127) / 128;

  if (tid == 0) {
    prefetch_map(&maps.a);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.acc_full[i], 1);
      mbar_init(&S.acc_empty[i], 2 * kAddWarps);
    }
    for (int i = 0; i < kScaleStages; ++i) {
      mbar_init(&S.sx_full[i], kScaleWarps);
      mbar_init(&S.sx_empty[i], kAddWarps);
    }
    mbar_init(&S.top_full, 2 * kAddWarps);
    mbar_init(&S.inverse_full, kAddWarps);
    S.waits.abort = 0;
    S.waits.limit = p.limit;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<true>(&S.tmem, 2 * kAccCols);
  pdl_wait();
  pdl_trigger();
  if (warp == 0) list_tiles<kFeat>(S, p.offsets, p.E, p.m, feats);
  fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised
  fence_after();
  const uint32_t tmem = S.tmem;
  const int t0 = blockIdx.x >> 1, stride = gridDim.x >> 1;
  int e = 0;
  Tile T;

  if (warp < 4) {
    give_registers<kFewRegs>();
    if (warp == 0) {
      if (elect_one()) {
        const uint32_t lead_full = map_rank(smem_u32(S.full), 0);
        int it = 0;
        bool go = true;
        for (int t = t0; go && tile_at<kFeat>(S, p.E, feats, t, e, T); t += stride) {
          const int half = T.n / 2;
          for (int b = 0; b < blocks; ++b, ++it) {
            const int s = it % kStages;
            if (!(go = it < p.stall && wait_bar(&S.empty[s], ((it / kStages) & 1) ^ 1, &S.waits))) break;
            if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2 * (kHalf + half * 128));
            const uint32_t a = smem_u32(S.stage[s]), bar = lead_full + 8 * s;
            if (kGated)
              load_5d<true>(a, &maps.a, 128 * b, 0, 0, (T.f0 + 64 * static_cast<int>(rank)) / 16, T.e, bar);
            else
              load_3d<true>(a, &maps.a, 128 * b, T.f0 + 128 * rank, T.e, bar);
            load_2d<true>(a + kHalf, &maps.b[half / 16 - 1], 128 * b, T.c0 + rank * half, bar);
          }
        }
      }
    } else if (warp == 1) {
      if (rank == 0 && elect_one()) {
        int it = 0;
        bool go = true;
        for (int t = t0; go && tile_at<kFeat>(S, p.E, feats, t, e, T); t += stride) {
          const uint32_t idesc = instr_desc8(256, T.n);
          for (int b = 0; b < blocks; ++b, ++it) {
            const int s = it % kStages, buf = it & 1;
            if (!(go = wait_bar(&S.acc_empty[buf], ((it >> 1) & 1) ^ 1, &S.waits) &&
                       wait_bar(&S.full[s], (it / kStages) & 1, &S.waits)))
              break;
            fence_after();
            const uint64_t da = tile_desc<false>(smem_u32(S.stage[s])), db = tile_desc<false>(smem_u32(S.stage[s]) + kHalf);
            const int steps = (min(128, p.k - 128 * b) + 31) / 32;
            for (int i = 0; i < steps; ++i)
              mma8_pair(tmem + buf * kAccCols, da + 2 * i, db + 2 * i, idesc, i != 0);
            commit_pair(&S.empty[s], 3);
            commit_pair(&S.acc_full[buf], 3);
          }
        }
      }
    }
  } else if (warp < 4 + kAddWarps) {
    take_registers<kManyRegs>();
    const int q = warp & 3, half = (warp - 4) >> 2;   // this warp's lanes of tensor memory; its 32 columns of each 64
    const uint32_t lead_empty = map_rank(smem_u32(S.acc_empty), 0), buf16 = smem_u32(S.epi[warp - 4]);
    const int rows_w = (p.n + 127) / 128;   // blocks of weight rows
    int it = 0, n_sx = 0, n_tile = 0;
    bool ok = true;
    for (int t = t0; ok && tile_at<kFeat>(S, p.E, feats, t, e, T); t += stride, ++n_tile) {
      // first feature of this warp's 32 lanes (gated: 16 gate and 16 up lanes of 16 features)
      const int f0 = T.f0 + (kGated ? 64 * static_cast<int>(rank) + 16 * q : 128 * static_cast<int>(rank) + 32 * q);
      const float* sw = p.sw + static_cast<long long>(T.e) * rows_w * blocks;
      RowScales s0{sw + min(f0 / 128, rows_w - 1) * blocks, 0.f};
      RowScales s1{sw + min((feats + f0) / 128, rows_w - 1) * blocks, 0.f};
      uint64_t acc[4][2][8];   // of 32 columns: 16 accumulator lanes each, pairs of columns
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][h][j] = 0;
      for (int b = 0; b < blocks; ++b, ++it) {
        const int buf = it & 1, sb = b % kScaleBlocks, ss = n_sx % kScaleStages;
        if (sb == 0 && !(ok = wait_bar_warp(&S.sx_full[ss], (n_sx / kScaleStages) & 1, &S.waits))) break;
        const float w0 = s0.at(b, blocks, lane), w1 = kGated ? s1.at(b, blocks, lane) : w0;
        const uint64_t w0x2 = pack_f32x2(w0, w0), w1x2 = pack_f32x2(w1, w1);
        if (!(ok = wait_bar_warp(&S.acc_full[buf], (it >> 1) & 1, &S.waits))) break;
        fence_after();
        const float* sx = S.sx[ss][sb] + 32 * half + 2 * (lane & 3);
        const uint32_t at = tmem + buf * kAccCols + 32 * half + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (32 * half + 64 * i >= T.cols) break;
          float v[2][16];
          ld_frags(at + 64 * i, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t x2 = *reinterpret_cast<const uint64_t*>(sx + 64 * i + 8 * j);
            const uint64_t g = mul_f32x2(x2, w0x2), u = kGated ? mul_f32x2(x2, w1x2) : g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              fma_f32x2(acc[i][h][2 * j], pack_f32x2(v[h][4 * j], v[h][4 * j + 1]), h ? u : g);
              fma_f32x2(acc[i][h][2 * j + 1], pack_f32x2(v[h][4 * j + 2], v[h][4 * j + 3]), h ? u : g);
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_cluster(lead_empty + 8 * buf);
          if (sb == kScaleBlocks - 1 || b == blocks - 1) mbarrier_arrive(&S.sx_empty[ss]);
        }
        if (sb == kScaleBlocks - 1 || b == blocks - 1) ++n_sx;
      }
      if (!ok) break;
      const int left = feats - f0;   // none or less: the output ends before this warp's features do
      if constexpr (kGated) {
        // a in the gate values' place, and its largest magnitude in each column
        uint32_t* mine = S.top[n_tile & 1][rank][q];
        const uint32_t other = map_rank(smem_u32(mine), rank ^ 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (32 * half + 64 * i >= T.cols) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t top[2] = {0, 0};
#pragma unroll
            for (int r = 0; r < 2; ++r) {   // features lane / 4 and lane / 4 + 8
              const uint64_t g = acc[i][0][2 * j + r], u = acc[i][1][2 * j + r];
              const float a0 = gelu16(lo_f32(g), p.gelu) * lo_f32(u), a1 = gelu16(hi_f32(g), p.gelu) * hi_f32(u);
              acc[i][0][2 * j + r] = pack_f32x2(a0, a1);
              if (left > 0) top[0] = max(top[0], abs_bits(a0)), top[1] = max(top[1], abs_bits(a1));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top[c] = max(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], d));
              if (lane < 4) {
                const int col = 32 * half + 64 * i + 8 * j + 2 * lane + c;
                mine[col] = top[c];
                st_cluster_u32(other + 4 * col, top[c]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          arrive_release_cluster(map_rank(smem_u32(&S.top_full), 0));
          arrive_release_cluster(map_rank(smem_u32(&S.top_full), 1));
        }
        bool met = try_wait_cluster(&S.top_full, n_tile & 1);
        for (const long long began = clock64(); !met && !S.waits.abort; met = try_wait_cluster(&S.top_full, n_tile & 1))
          if (clock64() - began > 1024LL * S.waits.limit) S.waits.abort = 1;
        if (!(ok = __all_sync(0xFFFFFFFFu, met))) break;
        const int col = (warp - 4) * 32 + lane;
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) top = max(top, S.top[n_tile & 1][r >> 2][r & 3][col]);
        const Scale8 sc = scale8(top);
        float* inverse = S.inverse[n_tile & 1];   // in turn: who writes one again knows that all have come to the tile between
        inverse[col] = sc.inverse;
        if (rank == 0 && col < T.cols)
          p.sa[static_cast<long long>(T.c0 + col) * ((feats + 127) / 128) + T.f0 / 128] = sc.scale;
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&S.inverse_full);
        if (!(ok = wait_bar_warp(&S.inverse_full, n_tile & 1, &S.waits))) break;
        uint8_t* out = static_cast<uint8_t*>(p.y) + f0;
        uint8_t* stage = S.epi[warp - 4];   // [32 columns][16 features], 16 bytes apart
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c0 = 32 * half + 64 * i;
          if (c0 >= T.cols) break;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t inv = *reinterpret_cast<const uint64_t*>(inverse + c0 + 8 * j + 2 * (lane & 3));
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint64_t v = mul_f32x2(acc[i][0][2 * j + r], inv);
              const uint32_t two = to_e4m3x2(lo_f32(v), hi_f32(v));
              const int at = (8 * j + 2 * (lane & 3)) * 16 + (lane >> 2) + 8 * r;
              stage[at] = static_cast<uint8_t>(two), stage[at + 16] = static_cast<uint8_t>(two >> 8);
            }
          }
          __syncwarp();
          if (c0 + lane < T.cols && left > 0)
            *reinterpret_cast<uint4*>(out + (T.c0 + c0 + lane) * p.ldy) = *reinterpret_cast<const uint4*>(stage + 16 * lane);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c0 = 32 * half + 64 * i, cols = T.cols - c0;
          if (cols <= 0) break;
          float v[2][16];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[h][2 * j] = lo_f32(acc[i][h][j]), v[h][2 * j + 1] = hi_f32(acc[i][h][j]);
          if (p.out == MOE_F32) {
            float* out = static_cast<float*>(p.y) + (T.c0 + c0) * p.ldy + f0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int c = 8 * j + 2 * (lane & 3) + (r & 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int f = 16 * h + 8 * (r >> 1) + (lane >> 2);
                  if (c < cols && f < left) out[c * p.ldy + f] = v[h][4 * j + r];
                }
              }
          } else {
            store_32x32(buf16, v, p.out == MOE_BF16, static_cast<uint16_t*>(p.y) + (T.c0 + c0) * p.ldy + f0, p.ldy, cols, left, lane);
          }
        }
      }
    }
  } else {
    give_registers<kFewRegs>();
    const int i0 = tid - 32 * (4 + kAddWarps);   // this thread turns the scales of rows i0 and i0 + 128
    int n_sx = 0;
    bool ok = true;
    for (int t = t0; ok && tile_at<kFeat>(S, p.E, feats, t, e, T); t += stride) {
      const float* from0 = p.sx + static_cast<long long>(min(T.c0 + min(i0, T.cols - 1), p.m - 1)) * blocks;
      const float* from1 = p.sx + static_cast<long long>(min(T.c0 + min(i0 + 128, T.cols - 1), p.m - 1)) * blocks;
      for (int b0 = 0; b0 < blocks; b0 += kScaleBlocks, ++n_sx) {
        float v[kScaleBlocks][2];
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) {
          const int b = min(b0 + i, blocks - 1);
          v[i][0] = from0[b];
          v[i][1] = from1[b];
        }
        const int ss = n_sx % kScaleStages;
        if (!(ok = wait_bar_warp(&S.sx_empty[ss], ((n_sx / kScaleStages) & 1) ^ 1, &S.waits))) break;
#pragma unroll
        for (int i = 0; i < kScaleBlocks; ++i) S.sx[ss][i][i0] = v[i][0], S.sx[ss][i][i0 + 128] = v[i][1];
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&S.sx_full[ss]);
      }
    }
  }
  fence_before();
  __syncthreads();
  if (S.waits.abort == 1) report_and_settle();
  cluster_sync();   // no CTA leaves while the other may still arrive on its barriers or read its stages
  fence_after();
  if (warp == 1) tmem_free<true>(tmem, 2 * kAccCols);
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

// [E][2][f][k] seen as blocks of 16 features: 16 gate and the same 16 up rows of four blocks.
bool map_gated8(CUtensorMap* m, const void* base, int E, int f, int k) {
  const cuuint64_t row = static_cast<cuuint64_t>(k);
  const cuuint64_t dim[5] = {row, 16, 2, static_cast<cuuint64_t>(f / 16), static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[4] = {row, row * f, row * 16, row * 2 * f};
  const cuuint32_t box[5] = {128, 16, 2, 4, 1};
  return encode_byte_tiles(m, base, 5, dim, stride, box);
}

template <bool kGated>
bool launch(const Maps8& maps, const Mm8Params& p, int sms, cudaStream_t s) {
  constexpr int kFeat = kGated ? 128 : 256;
  const int feats = kGated ? p.n / 2 : p.n;
  const long long most = (feats + kFeat - 1) / kFeat * (std::min(p.E, p.m) + static_cast<long long>(p.m) / 64);   // parts of 64
  const long long pairs = std::min<long long>(sms / 2, most);
  const size_t smem = sizeof(Smem8) + 1024;
  if (cudaFuncSetAttribute(k_grouped8<kGated>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_grouped8<kGated>, maps, p) == cudaSuccess;
}

}  // namespace

bool launch_grouped8(bool gated, const Mm8Params& params, cudaStream_t s) {
  Mm8Params p = params;
  const WaitLimits l = wait_limits();
  p.limit = l.cycles1024, p.stall = l.loads;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  Maps8 maps;
  const int largest = ((std::min(p.m, 256) + 31) & ~31) / 32;   // half of a tile's rows a CTA, in steps of 16
  for (int i = 0; i < largest; ++i)
    if (!map_rows8(&maps.b[i], p.x, p.k, p.m, p.ldx, 16 * (i + 1))) return false;
  if (!(gated ? map_gated8(&maps.a, p.w, p.E, p.n / 2, p.k) : map_weights8(&maps.a, p.w, p.E, p.n, p.k))) return false;
  return gated ? launch<true>(maps, p, sms, s) : launch<false>(maps, p, sms, s);
}

bool mm8_gave_up(cudaStream_t s, uint32_t* count) {
  return cudaMemcpyFromSymbolAsync(count, g_gave_up, sizeof(*count), 0, cudaMemcpyDeviceToHost, s) == cudaSuccess;
}

}  // namespace moe
