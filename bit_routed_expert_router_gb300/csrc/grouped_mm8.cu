// Products of e4m3 rows grouped by expert with e4m3 weights, scales for blocks
// of 128 of the reduction on both sides:
//
//   y[r, n] = sum_b sx[r, b] sw[e][n / 128, b] sum_{k in b} x[r, k] w[e][n, k]
//
// Each block of 128 is summed by itself in fp32, then scaled and added in fp32.
#include <algorithm>

#include "gelu16.cuh"
#include "moe.h"
#include "ops8.h"
#include "quant8.cuh"

namespace moe {

namespace {

constexpr int kRows = 8;   // of a tile

struct Tile8 {
  int e, row0, rows;
};

// Tile `index` of the groups cut into parts of kRows rows; rows = 0: there is none.  A group starts no earlier than the one
// before it ends and lies inside [0, m], whatever the offsets hold.
__device__ Tile8 find_tile(const int32_t* offsets, int E, int m, int index) {
  int lo = min(max(offsets[0], 0), m);
  for (int e = 0; e < E; ++e) {
    const int hi = max(lo, min(max(offsets[e + 1], 0), m)), n = (hi - lo + kRows - 1) / kRows;
    if (index < n) return {e, lo + index * kRows, min(kRows, hi - lo - index * kRows)};
    index -= n;
    lo = hi;
  }
  return {0, 0, 0};
}

// part[r] = sum over a block of 128 (or what is left of it) of row r's values in shared memory times a weight row's
__device__ void block_products(float (&part)[kRows], const uint8_t* w, int left, const float (&xs)[kRows][128]) {
  for (int r = 0; r < kRows; ++r) part[r] = 0.f;
  for (int c = 0; c < left; c += 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(w + c);
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = from_e4m3x2(word[i >> 1] >> (16 * (i & 1)));
#pragma unroll
      for (int r = 0; r < kRows; ++r) part[r] = fmaf(f.y, xs[r][c + 2 * i + 1], fmaf(f.x, xs[r][c + 2 * i], part[r]));
    }
  }
}

// 128 features x kRows rows a CTA, a feature a thread.
template <bool kGated>
__global__ void __launch_bounds__(128) k_grouped8(Mm8Params p) {
  __shared__ float xs[kRows][128];
  __shared__ Tile8 s_tile;
  __shared__ uint32_t s_top[4][kRows];
  if (threadIdx.x == 0) s_tile = find_tile(p.offsets, p.E, p.m, blockIdx.x);
  __syncthreads();
  const Tile8 T = s_tile;
  if (T.rows == 0) return;
  const int feats = kGated ? p.n / 2 : p.n, f = 128 * blockIdx.y + threadIdx.x, kb = (p.k + 127) / 128;
  const int nb = (p.n + 127) / 128, fr = min(f, feats - 1);
  const long long up = kGated ? feats : 0;
  const uint8_t* w = p.w + (static_cast<long long>(T.e) * p.n + fr) * p.k;
  const float* sw = p.sw + static_cast<long long>(T.e) * nb * kb;
  float g[kRows] = {}, u[kRows] = {};
  for (int b = 0; b < kb; ++b) {
    const int left = min(128, p.k - 128 * b);
    __syncthreads();
    for (int r = 0; r < kRows; ++r)
      if (static_cast<int>(threadIdx.x) < left)
        xs[r][threadIdx.x] = from_e4m3x2(p.x[(T.row0 + min(r, T.rows - 1)) * p.ldx + 128 * b + threadIdx.x]).x;
    __syncthreads();
    float part[kRows];
    block_products(part, w + 128 * b, left, xs);
    for (int r = 0; r < kRows; ++r)
      g[r] = fmaf(part[r], p.sx[static_cast<long long>(T.row0 + min(r, T.rows - 1)) * kb + b] * sw[fr / 128 * kb + b], g[r]);
    if (kGated) {
      block_products(part, w + up * p.k + 128 * b, left, xs);
      for (int r = 0; r < kRows; ++r)
        u[r] = fmaf(part[r], p.sx[static_cast<long long>(T.row0 + min(r, T.rows - 1)) * kb + b] * sw[(fr + up) / 128 * kb + b], u[r]);
    }
  }
  if (kGated) {
    for (int r = 0; r < kRows; ++r) {
      g[r] = gelu16(g[r], p.gelu) * u[r];
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, f < feats ? abs_bits(g[r]) : 0);
      if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5][r] = top;
    }
    __syncthreads();
    for (int r = 0; r < T.rows; ++r) {
      const Scale8 s = scale8(max(max(s_top[0][r], s_top[1][r]), max(s_top[2][r], s_top[3][r])));
      if (f < feats) static_cast<uint8_t*>(p.y)[(T.row0 + r) * p.ldy + f] = to_e4m3x2(g[r] * s.inverse, 0.f);
      if (threadIdx.x == 0) p.sa[static_cast<long long>(T.row0 + r) * ((feats + 127) / 128) + blockIdx.y] = s.scale;
    }
    return;
  }
  if (f < feats)
    for (int r = 0; r < T.rows; ++r) {
      const long long at = (T.row0 + r) * p.ldy + f;
      if (p.out == MOE_F32)
        static_cast<float*>(p.y)[at] = g[r];
      else if (p.out == MOE_BF16)
        static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(g[r]);
      else
        static_cast<__half*>(p.y)[at] = __float2half_rn(g[r]);
    }
}

}  // namespace

bool launch_grouped8(bool gated, const Mm8Params& p, cudaStream_t s) {
  const int feats = gated ? p.n / 2 : p.n, tiles = std::min(p.E, p.m) + p.m / kRows;
  const dim3 grid(tiles, (feats + 127) / 128);
  if (gated)
    k_grouped8<true><<<grid, 128, 0, s>>>(p);
  else
    k_grouped8<false><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace moe
