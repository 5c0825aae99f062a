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
//
// 4096 rows of 2816, delta in 16 bits, out in 8 bits: 15.3 us, 5.3 TB/s (78 % of a
// copy's rate).  Their gradient with dres: 19.7 us, of which 16.0 are the rows'
// (5.7 TB/s) and the rest the sum of the weight gradient's parts after them.  One
// row: 1.7 us in a graph, a launch.
#include <algorithm>

#include "allow_smem.h"
#include "f32x2.cuh"
#include "ops8.h"
#include "quant8.cuh"

namespace moe {

namespace {

// Eight values as four pairs: the arithmetic on them is two values an instruction (f32x2).
struct Eight {
  uint64_t p[4];
  __device__ __forceinline__ float lo(int i) const { return lo_f32(p[i]); }
  __device__ __forceinline__ float hi(int i) const { return hi_f32(p[i]); }
};

__device__ __forceinline__ uint64_t both(float v) { return pack_f32x2(v, v); }
__device__ __forceinline__ float sum2(uint64_t v) { return lo_f32(v) + hi_f32(v); }

template <bool kBf16>
__device__ __forceinline__ Eight widen(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  Eight o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o.p[i] = kBf16 ? pack_f32x2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)) : pack_f32x2(half_lo(w[i]), half_hi(w[i]));
  return o;
}

template <bool kBf16>
__device__ __forceinline__ uint4 narrow(const Eight& v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.lo(i), v.hi(i));
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __half2 p = __floats2half2_rn(v.lo(i), v.hi(i));
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

// 8-bit quotients come from u = r w: the product of two 16-bit values is exact.  Of bf16 the power of two in rstd goes into r
// first: u is then within a factor of two of v and leaves fp32's range only where v does (r w alone for rows of 1e17 and weights
// of 1e25; 4096 rows of 2816 15.0 -> 15.3 us).  The rest of rstd is in the scale, and cancels from the quotients where the largest |u| of a group is a top of
// common size.  With the roundings of 448 / top and of the product only, fewer of them land on the wrong side of a tie (of 78
// million values 8,700 instead of 14,300 differ from quotients in 64 bits, which break the exact ties among them as they come; as
// fp32 quotients of v and its scale 10,500).
constexpr float kLargest = 3.4028234663852886e38f;   // fp32's largest value

__device__ __forceinline__ bool common(float top) {
  constexpr uint32_t lo = 0x15000000u, hi = 0x6A000000u;   // 2^-85 and 2^85
  return __float_as_uint(top) - lo < hi - lo;
}

// 448 / top: the fast reciprocal after one of Newton's steps.
__device__ __forceinline__ float inverse_of(float top) {
  float x;
  asm("rcp.approx.f32 %0, %1;" : "=f"(x) : "f"(top));
  return kMaxE4m3 * fmaf(x, fmaf(-top, x, 1.f), x);
}

enum { kNoDelta = 0, kDelta16 = 1, kDelta32 = 2 };

// A row is the threads of one threadIdx.y; kV words of eight values a thread, of kR rows at a time: one barrier for all of them,
// and more loads on their way (4096 rows of 2816, 8-bit out: 15.0 us against 16.2).
template <bool kBf16, int kDelta, int kV, int kR>
__global__ void __launch_bounds__(kR == 2 ? 512 : 1024, kR == 2 ? 3 : 1) k_norm(NormParams p) {   // (with 52 registers 16.2 us)
  __shared__ float s_sum[kR][32];
  const int n_words = p.d / 8, warps = blockDim.x / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r0 = (blockIdx.x * blockDim.y + threadIdx.y) * kR;
  pdl_wait();
  pdl_trigger();
  Eight v[kR][kV];
  float sum[kR];
  uint4 w[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
    uint4 h[kR], d16[kR];
    float4 d32[kR][2];
#pragma unroll
    for (int q = 0; q < kR; ++q) {
      const int r = r0 + q;
      if (r < p.m && i < n_words) {
        h[q] = *reinterpret_cast<const uint4*>(row16(p.h, p.ldh, r, c));
        if (kDelta == kDelta16) d16[q] = *reinterpret_cast<const uint4*>(row16(p.delta, p.ldd, r, c));
        if (kDelta == kDelta32) {
          const float4* at = reinterpret_cast<const float4*>(static_cast<const float*>(p.delta) + r * p.ldd + c);
          d32[q][0] = at[0], d32[q][1] = at[1];
        }
      }
    }
    w[j] = p.weight && i < n_words ? __ldg(reinterpret_cast<const uint4*>(p.weight) + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < kR; ++q) {
      const int r = r0 + q;
      if (r < p.m && i < n_words) {
        v[q][j] = widen<kBf16>(h[q]);
        if (kDelta != kNoDelta) {
          Eight d;
          if (kDelta == kDelta16) {
            d = widen<kBf16>(d16[q]);
          } else {
            const float4 a = d32[q][0], b = d32[q][1];
            d = {{pack_f32x2(a.x, a.y), pack_f32x2(a.z, a.w), pack_f32x2(b.x, b.y), pack_f32x2(b.z, b.w)}};
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) v[q][j].p[k] = add_f32x2(v[q][j].p[k], d.p[k]);
          const uint4 stored = narrow<kBf16>(v[q][j]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.h_out) + r * p.ldo + c) = stored;
          v[q][j] = widen<kBf16>(stored);
        }
      } else {
        v[q][j] = {};
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kR; ++q) {
    uint64_t two = 0;
#pragma unroll
    for (int j = 0; j < kV; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) fma_f32x2(two, v[q][j].p[k], v[q][j].p[k]);
    sum[q] = warp_sum(sum2(two));
  }
  if (warps > 1) {
    const int mine = threadIdx.y * warps;
    if (lane == 0)
#pragma unroll
      for (int q = 0; q < kR; ++q) s_sum[q][mine + warp] = sum[q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kR; ++q) sum[q] = warp_sum(lane < warps ? s_sum[q][mine + lane] : 0.f);
  }
#pragma unroll
  for (int q = 0; q < kR; ++q) {
    const int r = r0 + q;
    const float rstd = rsqrtf(fmaf(sum[q], p.over_d, p.eps));
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + j * blockDim.x, c = 8 * i;
      const bool in = r < p.m && i < n_words;
      const auto f = [&](int k) { return widen<kBf16>(w[j]).p[k]; };
      if (p.y && in) {
        Eight y;
#pragma unroll
        for (int k = 0; k < 4; ++k) y.p[k] = mul_f32x2(v[q][j].p[k], both(rstd));
        if (p.weight)
#pragma unroll
          for (int k = 0; k < 4; ++k) y.p[k] = mul_f32x2(y.p[k], f(k));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + r * p.ldy + c) = narrow<kBf16>(y);
      }
      if (p.y8) {
        float rest = rstd;
        if (kBf16) {   // rstd = power * rest, 1 <= rest < 2 (an rstd of 0, infinity or NaN is all in power); of fp16 |r w| is in range
          const float power = rstd < kLargest ? __uint_as_float(__float_as_uint(rstd) & 0x7F800000u) : rstd;
          rest = __uint_as_float((__float_as_uint(rstd) & 0x007FFFFFu) | 0x3F800000u);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[q][j].p[k] = mul_f32x2(v[q][j].p[k], both(power));
        }
        if (p.weight)
#pragma unroll
          for (int k = 0; k < 4; ++k) v[q][j].p[k] = mul_f32x2(v[q][j].p[k], f(k));
        float top = 0.f;   // of the 16 lanes that hold a group; words past the row are 0
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max_abs(max_abs(top, v[q][j].lo(k)), v[q][j].hi(k));
#pragma unroll
        for (int d = 8; d; d >>= 1) top = max_abs(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        Scale8 s;
        const float least = max_abs(kTiny, top * rest);
        if (common(top) && least > kTiny) {
          s.scale = least * (1.f / kMaxE4m3);
          s.inverse = inverse_of(top);
        } else {   // the least scale, or values that are not finite
          s = scale8(least);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[q][j].p[k] = mul_f32x2(v[q][j].p[k], both(rest));
        }
        if (in) {
          Eight a;
#pragma unroll
          for (int k = 0; k < 4; ++k) a.p[k] = mul_f32x2(v[q][j].p[k], both(s.inverse));
          *reinterpret_cast<uint2*>(p.y8 + r * p.ldy8 + c) =
              make_uint2(to_e4m3x4(a.lo(0), a.hi(0), a.lo(1), a.hi(1)), to_e4m3x4(a.lo(2), a.hi(2), a.lo(3), a.hi(3)));
          if ((i & 15) == 0) p.scale[static_cast<long long>(r) * ((p.d + 127) / 128) + i / 16] = s.scale;
        }
      }
    }
  }
}

__device__ __forceinline__ void copy16(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Rows on their way to a CTA of k_norm_grad (4096 rows of 2816: two 20.0 us, three 20.2, four 21.0).
constexpr int kGradStages = 2;

// CTA b takes the rows b, b + parts, ...: its columns' part of the weight gradient stays in registers and is written once.  The
// next rows are on their way to shared memory, each thread's words to its own place there, which needs no barrier.  (With one
// row on its way in registers 22.0 us for 4096 rows of 2816, with none 36; with three CTAs an SM 20.5.)
template <bool kBf16, int kV, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads <= 512 ? 2 : 1) k_norm_grad(NormGradParams p) {
  constexpr int kStages = kGradStages;
  extern __shared__ uint4 s_rows[];   // [stage][h, dy, dres][word of a thread][thread]
  __shared__ float2 s_sum[2][32];
  const int n_words = p.d / 8, warps = blockDim.x / 32, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const auto place = [&](int s, int which, int j) { return s_rows + ((s * 3 + which) * kV + j) * blockDim.x + threadIdx.x; };
  const auto load = [&](int r, int s) {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i >= n_words || r >= p.m) continue;
      copy16(place(s, 0, j), row16(p.h, p.ldh, r, 8 * i));
      copy16(place(s, 1, j), row16(p.dy, p.lddy, r, 8 * i));
      if (p.dres) copy16(place(s, 2, j), row16(p.dres, p.lddres, r, 8 * i));
    }
    end_copies();
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) load(blockIdx.x + s * gridDim.x, s);
  // A row's values stay in registers between its sums and its outputs where a thread has one word of them; two would spill
  // (2000 rows of 5632 34.4 us, 700 of 16,384 39.9) or leave room for one CTA an SM (22.9 us, the former), so they are read
  // again, and the weight is kept as it is (21.4 and 24.4; all bf16 with dres).
  constexpr bool kAgain = kV > 1;
  Eight dw[kV], w[kV];
  uint4 w_raw[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    const uint32_t one = kBf16 ? 0x3F803F80u : 0x3C003C00u;
    w_raw[j] = p.weight && i < n_words ? __ldg(reinterpret_cast<const uint4*>(p.weight) + i) : make_uint4(one, one, one, one);
    w[j] = widen<kBf16>(w_raw[j]);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[j].p[k] = 0;
  }
  int turn = 0, s = 0;
  for (int r = blockIdx.x; r < p.m; r += gridDim.x, turn ^= 1) {
    Eight a[kV], b[kV], o[kV];
    uint64_t ss2 = 0, dot2 = 0;
    const auto fetch = [&](int j) {
      const uint4 none = make_uint4(0, 0, 0, 0);
      const bool in = static_cast<int>(threadIdx.x + j * blockDim.x) < n_words;
      a[j] = widen<kBf16>(in ? *place(s, 0, j) : none);
      b[j] = widen<kBf16>(in ? *place(s, 1, j) : none);
      o[j] = widen<kBf16>(in && p.dres ? *place(s, 2, j) : none);
      if (kAgain) w[j] = widen<kBf16>(w_raw[j]);
    };
    wait_copies<kStages - 1>();
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      fetch(j);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        fma_f32x2(ss2, a[j].p[k], a[j].p[k]);
        fma_f32x2(dot2, mul_f32x2(b[j].p[k], w[j].p[k]), a[j].p[k]);
      }
    }
    if (!kAgain) load(r + kStages * gridDim.x, s);
    float ss = warp_sum(sum2(ss2)), dot = warp_sum(sum2(dot2));
    if (warps > 1) {
      if (lane == 0) s_sum[turn][warp] = make_float2(ss, dot);
      __syncthreads();
      const float2 v = lane < warps ? s_sum[turn][lane] : make_float2(0.f, 0.f);
      ss = warp_sum(v.x);
      dot = warp_sum(v.y);
    }
    const float rstd = rsqrtf(fmaf(ss, p.over_d, p.eps));
    const float mean = rstd * (rstd * (dot * rstd * p.over_d));   // of dy w xh, times rstd^2
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (kAgain) fetch(j);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        fma_f32x2(dw[j].p[k], b[j].p[k], mul_f32x2(a[j].p[k], both(rstd)));
        uint64_t own = mul_f32x2(a[j].p[k], both(-mean));
        fma_f32x2(own, mul_f32x2(b[j].p[k], w[j].p[k]), both(rstd));
        o[j].p[k] = add_f32x2(o[j].p[k], own);
      }
      if (i < n_words) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dh) + r * p.lddh + 8 * i) = narrow<kBf16>(o[j]);
    }
    if (kAgain) load(r + kStages * gridDim.x, s);
    s = (s + 1) % kStages;
  }
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i >= n_words) continue;
    float4* at = reinterpret_cast<float4*>(p.part + static_cast<long long>(blockIdx.x) * p.d + 8 * i);
    at[0] = make_float4(dw[j].lo(0), dw[j].hi(0), dw[j].lo(1), dw[j].hi(1));
    at[1] = make_float4(dw[j].lo(2), dw[j].hi(2), dw[j].lo(3), dw[j].hi(3));
  }
}

// Sums of the columns of part [parts][d], in a fixed order: 32 columns a CTA, 64 threads for each four of them.
__global__ void __launch_bounds__(512) k_norm_dweight(const float* part, int parts, int d, float* dweight) {
  __shared__ float4 s_sum[64][8];
  const int q = threadIdx.x & 7, g = threadIdx.x >> 3, c = 32 * blockIdx.x + 4 * q;
  pdl_wait();
  pdl_trigger();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d)
#pragma unroll 8
    for (int i = g; i < parts; i += 64) {
      const float4 v = *reinterpret_cast<const float4*>(part + static_cast<long long>(i) * d + c);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
  s_sum[g][q] = sum;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // 32 columns, one a thread
  const float* col = reinterpret_cast<const float*>(s_sum) + threadIdx.x;
  float total = 0.f;
#pragma unroll 16
  for (int i = 0; i < 64; ++i) total += col[32 * i];
  if (32 * blockIdx.x + threadIdx.x < d) dweight[32 * blockIdx.x + threadIdx.x] = total;
}

template <typename K, typename... A>
bool launch(K kernel, dim3 grid, dim3 block, cudaStream_t s, int smem, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <bool kBf16, int kDelta, int kV, int kR>
bool launch_rows(const NormParams& p, int nt, int rows, cudaStream_t s) {
  return launch(k_norm<kBf16, kDelta, kV, kR>, dim3((p.m + rows * kR - 1) / (rows * kR)), dim3(nt, rows), s, 0, p);
}

template <bool kBf16, int kDelta>
bool launch_norm_of(const NormParams& p, int sms, cudaStream_t s) {
  const int words = p.d / 8;
  if (words > 1024) return launch_rows<kBf16, kDelta, 2, 1>(p, 1024, 1, s);
  const int nt = (words + 31) / 32 * 32, rows = std::max(1, 256 / nt);
  // Two rows a thread where that leaves every SM two CTAs of long rows (2816 values: 600 rows 3.1 us either way, 2400 10.0 against
  // 10.7, 300 2.4 against 2.3) or eight of short ones (264 values: 20,000 rows 10.8 us against 11.5, 9000 5.5 against 5.4, 4000
  // 4.3 against 3.4).  Not with fp32 delta, whose words take twice the registers (4096 rows of 2816, 16-bit out, 20.9 us, with two
  // rows that spill 26.1, with two rows and two CTAs an SM 24.4; 20,000 of 264 13.9, 17.0 and 14.9).
  if constexpr (kDelta != kDelta32)
    if (nt <= 512 && p.m >= (rows == 1 ? 4 : 16) * rows * sms) return launch_rows<kBf16, kDelta, 1, 2>(p, nt, rows, s);
  return launch_rows<kBf16, kDelta, 1, 1>(p, nt, rows, s);
}

template <bool kBf16, int kV, int kThreads>
bool launch_grad_rows(const NormGradParams& p, int nt, cudaStream_t s) {
  constexpr int kMost = kGradStages * 3 * kV * kThreads * 16;
  return allow_smem(k_norm_grad<kBf16, kV, kThreads>, kMost) &&
         launch(k_norm_grad<kBf16, kV, kThreads>, dim3(p.parts), dim3(nt), s, kGradStages * 3 * kV * nt * 16, p);
}

template <bool kBf16>
bool launch_grad_of(const NormGradParams& p, cudaStream_t s) {
  const int words = p.d / 8, nt = (words + 31) / 32 * 32;
  if (nt <= 512) return launch_grad_rows<kBf16, 1, 512>(p, nt, s);
  const int half = (words + 63) / 64 * 32;   // two words a thread
  return half <= 512 ? launch_grad_rows<kBf16, 2, 512>(p, half, s) : launch_grad_rows<kBf16, 2, 1024>(p, half, s);
}

// Multiprocessors of the current device; 0: a CUDA call failed.
int multiprocessors() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

}  // namespace

bool launch_norm(bool bf16, bool delta_f32, const NormParams& params, cudaStream_t s) {
  NormParams p = params;
  p.over_d = 1.f / static_cast<float>(p.d);
  const int sms = multiprocessors();
  if (!sms) return false;
  if (!p.delta) return bf16 ? launch_norm_of<true, kNoDelta>(p, sms, s) : launch_norm_of<false, kNoDelta>(p, sms, s);
  if (delta_f32) return bf16 ? launch_norm_of<true, kDelta32>(p, sms, s) : launch_norm_of<false, kDelta32>(p, sms, s);
  return bf16 ? launch_norm_of<true, kDelta16>(p, sms, s) : launch_norm_of<false, kDelta16>(p, sms, s);
}

bool launch_norm_grad(bool bf16, const NormGradParams& params, cudaStream_t s) {
  NormGradParams p = params;
  p.over_d = 1.f / static_cast<float>(p.d);
  const int sms = multiprocessors();
  if (!sms) return false;
  // all CTAs at once: two an SM, or one of 1024 threads; more where a row is few warps
  const int words = p.d / 8, warps = words > 512 ? (words + 63) / 64 : (words + 31) / 32;
  p.parts = std::min({p.m, kNormParts, sms * std::max(1, 32 / warps)});
  if (!(bf16 ? launch_grad_of<true>(p, s) : launch_grad_of<false>(p, s))) return false;
  return !p.part || launch(k_norm_dweight, dim3((p.d + 31) / 32), dim3(512), s, 0, static_cast<const float*>(p.part), p.parts,
                           p.d, p.dweight);
}

}  // namespace moe
