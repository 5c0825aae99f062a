// Root-mean-square norm with the residual's addition, and its gradient.
//
//   r = round16(h + delta)    v = r rstd w,  rstd = 1 / sqrt(mean(r^2) + eps)
//   y = round16(v)            y8, scale: v in e4m3, a scale for each 128 values
//   dh = dres + rstd (dy w - xh mean(dy w xh)),  xh = r rstd
//   dw = sum over the rows of dy xh
//
// Sums are fp32.  The stored r is what is normalised, so that the gradient and
// the next layer, which read it, see the same values.  Memory-bound: every
// value is read once, a row stays in registers between its sum and its outputs,
// eight values (16 bytes) a thread.
#include <algorithm>

#include "ops8.h"
#include "quant8.cuh"

namespace moe {

namespace {

template <bool kBf16>
__device__ __forceinline__ void widen(float (&o)[8], uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = kBf16 ? __uint_as_float(w[i] << 16) : half_lo(w[i]);
    o[2 * i + 1] = kBf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : half_hi(w[i]);
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ const uint16_t* row16(const void* p, long long ld, int r, int c) {
  return static_cast<const uint16_t*>(p) + r * ld + c;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

enum { kNoDelta = 0, kDelta16 = 1, kDelta32 = 2 };

// A row is the threads of one threadIdx.y; kV words of eight values a thread.
template <bool kBf16, int kDelta, int kV>
__global__ void __launch_bounds__(1024) k_norm(NormParams p) {
  __shared__ float s_sum[32];
  const int r = blockIdx.x * blockDim.y + threadIdx.y, n_words = p.d / 8, warps = blockDim.x / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool in_row = r < p.m;
  pdl_wait();
  pdl_trigger();
  float v[kV][8], sum = 0.f;
  uint4 w[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
    if (in_row && i < n_words) {
      const uint4 h = *reinterpret_cast<const uint4*>(row16(p.h, p.ldh, r, c));
      if (p.weight) w[j] = __ldg(reinterpret_cast<const uint4*>(p.weight) + i);
      widen<kBf16>(v[j], h);
      if (kDelta != kNoDelta) {
        float d[8];
        if (kDelta == kDelta16) {
          widen<kBf16>(d, *reinterpret_cast<const uint4*>(row16(p.delta, p.ldd, r, c)));
        } else {
          const float4* at = reinterpret_cast<const float4*>(static_cast<const float*>(p.delta) + r * p.ldd + c);
          const float4 a = at[0], b = at[1];
          d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += d[k];
        const uint4 stored = narrow<kBf16>(v[j]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h_out) + r * p.ldo + c) = stored;
        widen<kBf16>(v[j], stored);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(v[j][k], v[j][k], sum);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = 0.f;
    }
  }
  sum = warp_sum(sum);
  if (warps > 1) {
    float* mine = s_sum + threadIdx.y * warps;
    if (lane == 0) mine[warp] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < warps; ++i) sum += mine[i];
  }
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
    const bool in = in_row && i < n_words;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] *= rstd;
    if (p.weight && in) {
      float f[8];
      widen<kBf16>(f, w[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= f[k];
    }
    if (in && p.y) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + r * p.ldy + c) = narrow<kBf16>(v[j]);
    if (p.y8) {
      uint32_t top = 0;   // of the 16 lanes that hold a group; words past the row are 0
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, abs_bits(v[j][k]));
      if (!in) top = 0;
#pragma unroll
      for (int d = 8; d; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      const Scale8 s = scale8(top);
      if (in) {
        const float q = s.inverse;
        *reinterpret_cast<uint2*>(p.y8 + r * p.ldy8 + c) =
            make_uint2(to_e4m3x4(v[j][0] * q, v[j][1] * q, v[j][2] * q, v[j][3] * q),
                       to_e4m3x4(v[j][4] * q, v[j][5] * q, v[j][6] * q, v[j][7] * q));
        if ((i & 15) == 0) p.scale[static_cast<long long>(r) * ((p.d + 127) / 128) + i / 16] = s.scale;
      }
    }
  }
}

// CTA b takes the rows b, b + parts, ...: its columns' part of the weight gradient stays in registers and is written once.
template <bool kBf16, int kV>
__global__ void __launch_bounds__(1024) k_norm_grad(NormGradParams p) {
  __shared__ float2 s_sum[2][32];
  const int n_words = p.d / 8, warps = blockDim.x / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  float dw[kV][8];
  uint4 wt[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.f;
    if (p.weight && i < n_words) wt[j] = __ldg(reinterpret_cast<const uint4*>(p.weight) + i);
  }
  int turn = 0;
  for (int r = blockIdx.x; r < p.m; r += gridDim.x, turn ^= 1) {
    uint4 h[kV], dy[kV], dres[kV];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
      if (i >= n_words) continue;
      h[j] = *reinterpret_cast<const uint4*>(row16(p.h, p.ldh, r, c));
      dy[j] = *reinterpret_cast<const uint4*>(row16(p.dy, p.lddy, r, c));
      if (p.dres) dres[j] = *reinterpret_cast<const uint4*>(row16(p.dres, p.lddres, r, c));
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      if (threadIdx.x + j * blockDim.x >= n_words) continue;
      float a[8], b[8], w[8];
      widen<kBf16>(a, h[j]);
      widen<kBf16>(b, dy[j]);
      if (p.weight) widen<kBf16>(w, wt[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss = fmaf(a[k], a[k], ss);
        dot = fmaf(p.weight ? b[k] * w[k] : b[k], a[k], dot);
      }
    }
    ss = warp_sum(ss);
    dot = warp_sum(dot);
    if (warps > 1) {
      if (lane == 0) s_sum[turn][warp] = make_float2(ss, dot);
      __syncthreads();
      ss = dot = 0.f;
      for (int i = 0; i < warps; ++i) {
        const float2 v = s_sum[turn][i];
        ss += v.x;
        dot += v.y;
      }
    }
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.d) + p.eps);
    const float mean = dot * rstd / static_cast<float>(p.d);   // of dy w xh
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
      if (i >= n_words) continue;
      float a[8], b[8], w[8], o[8];
      widen<kBf16>(a, h[j]);
      widen<kBf16>(b, dy[j]);
      if (p.weight) widen<kBf16>(w, wt[j]);
      if (p.dres) widen<kBf16>(o, dres[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float xh = a[k] * rstd, g = p.weight ? b[k] * w[k] : b[k], dx = rstd * (g - xh * mean);
        dw[j][k] = fmaf(b[k], xh, dw[j][k]);
        o[k] = p.dres ? o[k] + dx : dx;
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dh) + r * p.lddh + c) = narrow<kBf16>(o);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i >= n_words) continue;
    float4* at = reinterpret_cast<float4*>(p.part + static_cast<long long>(blockIdx.x) * p.d + 8 * i);
    at[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
    at[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
  }
}

// Sums of the columns of part [parts][d], in a fixed order: 32 columns a CTA, 32 threads for each four of them.
__global__ void __launch_bounds__(256) k_norm_dweight(const float* part, int parts, int d, float* dweight) {
  __shared__ float4 s_sum[32][8];
  const int q = threadIdx.x & 7, g = threadIdx.x >> 3, c = 32 * blockIdx.x + 4 * q;
  pdl_wait();
  pdl_trigger();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d)
#pragma unroll 8
    for (int i = g; i < parts; i += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<long long>(i) * d + c);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
  s_sum[g][q] = sum;
  __syncthreads();
  if (g != 0 || c >= d) return;
  for (int i = 1; i < 32; ++i) {
    const float4 v = s_sum[i][q];
    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
  }
  *reinterpret_cast<float4*>(dweight + c) = sum;
}

template <typename K, typename... A>
bool launch(K kernel, dim3 grid, dim3 block, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <bool kBf16, int kDelta>
bool launch_norm_of(const NormParams& p, cudaStream_t s) {
  const int words = p.d / 8;
  if (words > 1024) return launch(k_norm<kBf16, kDelta, 2>, dim3(p.m), dim3(1024), s, p);
  const int nt = (words + 31) / 32 * 32, rows = std::max(1, 256 / nt);
  return launch(k_norm<kBf16, kDelta, 1>, dim3((p.m + rows - 1) / rows), dim3(nt, rows), s, p);
}

template <bool kBf16>
bool launch_grad_of(const NormGradParams& p, cudaStream_t s) {
  const int words = p.d / 8;
  return words > 1024 ? launch(k_norm_grad<kBf16, 2>, dim3(p.parts), dim3(1024), s, p)
                      : launch(k_norm_grad<kBf16, 1>, dim3(p.parts), dim3((words + 31) / 32 * 32), s, p);
}

}  // namespace

bool launch_norm(bool bf16, bool delta_f32, const NormParams& p, cudaStream_t s) {
  if (!p.delta) return bf16 ? launch_norm_of<true, kNoDelta>(p, s) : launch_norm_of<false, kNoDelta>(p, s);
  if (delta_f32) return bf16 ? launch_norm_of<true, kDelta32>(p, s) : launch_norm_of<false, kDelta32>(p, s);
  return bf16 ? launch_norm_of<true, kDelta16>(p, s) : launch_norm_of<false, kDelta16>(p, s);
}

bool launch_norm_grad(bool bf16, const NormGradParams& params, cudaStream_t s) {
  NormGradParams p = params;
  p.parts = std::min(p.m, kNormParts);
  if (!(bf16 ? launch_grad_of<true>(p, s) : launch_grad_of<false>(p, s))) return false;
  return !p.part || launch(k_norm_dweight, dim3((p.d + 31) / 32), dim3(256), s, static_cast<const float*>(p.part), p.parts,
                           p.d, p.dweight);
}

}  // namespace moe
