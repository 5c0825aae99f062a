// Kernels around the 16-bit grouped products: the gradient of the gated
// product, and the down half of the per-request adapters.
#include <algorithm>

#include "common.cuh"
#include "gelu16.cuh"
#include "grouped.h"

namespace moe {

namespace {

template <bool kBf16>
__device__ __forceinline__ float2 to_floats(uint32_t v) {
  if (kBf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  return make_float2(half_lo(v), half_hi(v));
}

template <bool kBf16>
__device__ __forceinline__ uint32_t to_pair(float a, float b) {
  if (kBf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// dh = [da u GELU'(g), da GELU(g)] for h = [g, u]: 16-byte loads and stores,
// eight features a thread.  Memory-bound: 10 bytes in and out per feature and
// about 30 operations; two words a thread were slower (41 us against 38 at
// 32,768 x 704).
template <bool kBf16, int kGelu>
__global__ void __launch_bounds__(256) k_gated_grad(const uint16_t* h, long long ldh, const uint16_t* da, long long ldda,
                                                    uint16_t* dh, long long lddh, int m, int f, const int32_t* n_rows) {
  pdl_wait();
  pdl_trigger();
  const int rows = n_rows ? min(*n_rows, m) : m, words = f / 8;
  const long long i = blockIdx.x * 256LL + threadIdx.x, r = i / words;
  if (r >= rows) return;
  const int c = static_cast<int>(i - r * words) * 8;
  const uint4 gv = *reinterpret_cast<const uint4*>(h + r * ldh + c);
  const uint4 uv = *reinterpret_cast<const uint4*>(h + r * ldh + f + c);
  const uint4 dv = *reinterpret_cast<const uint4*>(da + r * ldda + c);
  const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w}, d[4] = {dv.x, dv.y, dv.z, dv.w};
  uint32_t dg[4], du[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 gg = to_floats<kBf16>(g[w]), uu = to_floats<kBf16>(u[w]), dd = to_floats<kBf16>(d[w]);
    const float2 a = gelu16_and_slope<kGelu>(gg.x), b = gelu16_and_slope<kGelu>(gg.y);
    dg[w] = to_pair<kBf16>(dd.x * uu.x * a.y, dd.y * uu.y * b.y);
    du[w] = to_pair<kBf16>(dd.x * a.x, dd.y * b.x);
  }
  *reinterpret_cast<uint4*>(dh + r * lddh + c) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
  *reinterpret_cast<uint4*>(dh + r * lddh + f + c) = make_uint4(du[0], du[1], du[2], du[3]);
}

// ------------------------------------------------------------------ adapters: u = s A x

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kDownWarps = 16, kDownRows = 32;

// acc += A x for 16 rank rows and 8 kNg rows of x over the 64-value pieces k0,
// k0 + step, ... of the reduction.  A lane's fragments are 16 consecutive
// values of a row, loaded as two 16-byte words; the order of k inside a 64 is
// the same in both operands, which is all a product needs.  The next piece's
// loads are issued before this one's products.
template <bool kBf16, int kNg>
__device__ __forceinline__ void down_products(float (&acc)[4][4], const uint16_t* arow, bool has0, bool has1,
                                              const uint16_t* const (&xrow)[4], int k, int k0, int step, int t4) {
  struct Piece {
    uint4 a[2][2], x[kNg][2];
  };
  const auto load = [&](Piece& P, int at0) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int at = at0 + 16 * t4 + 8 * hh;
      const bool in = at < k;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      P.a[0][hh] = in && has0 ? __ldg(reinterpret_cast<const uint4*>(arow + at)) : zero;
      P.a[1][hh] = in && has1 ? __ldg(reinterpret_cast<const uint4*>(arow + 8 * static_cast<size_t>(k) + at)) : zero;
#pragma unroll
      for (int j = 0; j < kNg; ++j) P.x[j][hh] = in ? __ldg(reinterpret_cast<const uint4*>(xrow[j] + at)) : zero;
    }
  };
  const auto multiply = [&](const Piece& P) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t af[4] = {s ? P.a[0][hh].z : P.a[0][hh].x, s ? P.a[1][hh].z : P.a[1][hh].x,
                                s ? P.a[0][hh].w : P.a[0][hh].y, s ? P.a[1][hh].w : P.a[1][hh].y};
#pragma unroll
        for (int j = 0; j < kNg; ++j) {
          const uint32_t b0 = s ? P.x[j][hh].z : P.x[j][hh].x, b1 = s ? P.x[j][hh].w : P.x[j][hh].y;
          if (kBf16)
            mma_bf16(acc[j], af, b0, b1);
          else
            mma_f16(acc[j], af, b0, b1);
        }
      }
  };
  Piece a, b;   // three in flight were no faster
  load(a, k0);
  for (; k0 < k; k0 += 2 * step) {
    load(b, k0 + step);
    multiply(a);
    load(a, k0 + 2 * step);
    multiply(b);
  }
}

// A CTA: 16 rank rows x 32 rows of x, for the distinct adapters number z,
// z + gridDim.z, ... of those rows.  An adapter's rows are gathered, so that
// its products cost 8 rows at a time whatever their order.  The warps split
// the reduction and are added in order through shared memory.
template <bool kBf16>
__global__ void __launch_bounds__(32 * kDownWarps)
    k_adapter_down(const uint16_t* __restrict__ x, long long ldx, int t, const uint16_t* __restrict__ a,
                   const float* __restrict__ scale, const int32_t* __restrict__ ids, int n_adapters, int rank, int k,
                   float* u) {
  __shared__ float red[kDownWarps][16][kDownRows + 1];
  __shared__ uint8_t list[kDownWarps][kDownRows];   // a warp's own copy: the adapter's rows in order
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int row0 = blockIdx.x * kDownRows, r0 = blockIdx.y * 16;
  int id = -1;
  if (row0 + lane < t) {
    id = ids[row0 + lane];
    if (id < 0 || id >= n_adapters) id = -1;
  }
  uint32_t left = __ballot_sync(0xFFFFFFFFu, id >= 0);
  for (int nth = 0; left; ++nth) {
    const int ad = __shfl_sync(0xFFFFFFFFu, id, __ffs(left) - 1);
    const uint32_t same = __ballot_sync(0xFFFFFFFFu, id == ad);
    left &= ~same;
    if (nth % static_cast<int>(gridDim.z) != static_cast<int>(blockIdx.z)) continue;
    const int rows = __popc(same), groups = (rows + 7) / 8;
    __syncwarp();
    if (id == ad) list[warp][__popc(same & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane);
    __syncwarp();
    const float sc = scale[ad];
    const uint16_t* arow = a + (static_cast<size_t>(ad) * rank + r0 + g) * k;
    const uint16_t* xrow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)   // the last group repeats its last row
      xrow[j] = x + static_cast<long long>(row0 + list[warp][min(8 * j + g, rows - 1)]) * ldx;
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const bool has0 = r0 + g < rank, has1 = r0 + 8 + g < rank;
    const int k0 = 64 * warp, step = 64 * kDownWarps;
    if (groups == 1)
      down_products<kBf16, 1>(acc, arow, has0, has1, xrow, k, k0, step, t4);
    else if (groups == 2)
      down_products<kBf16, 2>(acc, arow, has0, has1, xrow, k, k0, step, t4);
    else
      down_products<kBf16, 4>(acc, arow, has0, has1, xrow, k, k0, step, t4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][g + 8 * (i >> 1)][8 * j + 2 * t4 + (i & 1)] = acc[j][i];
    __syncthreads();
    for (int i = tid; i < 16 * rows; i += 32 * kDownWarps) {
      const int r = i & 15, c = i >> 4;
      if (r0 + r >= rank) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kDownWarps; ++w) v += red[w][r][c];
      u[static_cast<size_t>(row0 + list[warp][c]) * rank + r0 + r] = v * sc;
    }
    __syncthreads();
  }
}

template <typename K, typename... A>
bool launch_pdl(K kernel, dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace

bool launch_gated_grad(bool bf16, int gelu, const void* h, long long ldh, const void* da, long long ldda, void* dh,
                       long long lddh, int m, int f, const int32_t* n_rows, cudaStream_t s) {
  const long long words = static_cast<long long>(m) * (f / 8);
  const dim3 grid(static_cast<unsigned>((words + 255) / 256));
  const auto kernel = bf16 ? (gelu == 1 ? k_gated_grad<true, 1> : k_gated_grad<true, 0>)
                           : (gelu == 1 ? k_gated_grad<false, 1> : k_gated_grad<false, 0>);
  return launch_pdl(kernel, grid, 256, s, static_cast<const uint16_t*>(h), ldh, static_cast<const uint16_t*>(da), ldda,
                    static_cast<uint16_t*>(dh), lddh, m, f, n_rows);
}

bool launch_adapter_down(bool bf16, const void* x, long long ldx, int t, const void* a, const float* scale,
                         const int32_t* ids, int n_adapters, int rank, int k, float* u, cudaStream_t s) {
  // a CTA for every 16 rank rows, and up to one for each distinct adapter of its 32 rows
  const int blocks = (t + kDownRows - 1) / kDownRows, parts = (rank + 15) / 16;
  const int shares = std::max(1, std::min({std::min(t, kDownRows), n_adapters, 512 / (blocks * parts)}));
  const auto kernel = bf16 ? k_adapter_down<true> : k_adapter_down<false>;
  return launch_pdl(kernel, dim3(blocks, parts, shares), 32 * kDownWarps, s, static_cast<const uint16_t*>(x), ldx, t,
                    static_cast<const uint16_t*>(a), scale, ids, n_adapters, rank, k, u);
}

}  // namespace moe
