// A routed layer and its shared expert for up to 32 tokens, in two kernels:
//
//   a[t, j] = gates[t, j] GELU(g) u,  [g, u] = Wgu[ids[t, j]] x[t]    rounded to the call's type
//   y[t] = sum_j Wd[ids[t, j]] a[t, j] + Wd_shared a_shared[t]
//
// A warp for each output value.
#include <algorithm>

#include "gelu16.cuh"
#include "ops8.h"
#include "quant8.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float value16(uint16_t v, int bf16) {
  return bf16 ? bf16_bits_to_float(v) : __half2float(__ushort_as_half(v));
}

// A warp's product of row `n` of a matrix [..][k] (of rows before it: `base`) with x, in every lane.
template <bool kW8>
__device__ float dot(const void* w, const float* scale, long long n, int k, const uint16_t* x, int bf16) {
  float sum = 0.f;
  for (int c = threadIdx.x & 31; c < k; c += 32) {
    float v;
    if (kW8)
      v = from_e4m3x2(static_cast<const uint8_t*>(w)[n * k + c]).x * scale[c / 128];
    else
      v = value16(static_cast<const uint16_t*>(w)[n * k + c], bf16);
    sum = fmaf(v, value16(x[c], bf16), sum);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  return sum;
}

// The scales of row n (of expert e) of matrices [rows][k].
__device__ __forceinline__ const float* scales(const float* s, long long e, int rows, int n, int k) {
  return s + (e * ((rows + 127) / 128) + n / 128) * ((k + 127) / 128);
}

template <bool kW8>
__global__ void __launch_bounds__(256) k_layer_up(LayerParams p) {
  const int pair = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5), pairs = p.t * p.k;
  const bool shared = pair >= pairs;
  const int t = shared ? pair - pairs : pair / p.k, f = shared ? p.fs : p.f, e = shared ? 0 : p.ids[pair];
  if (i >= f || e < 0 || e >= p.E) return;
  const FfnWeights& w = shared ? p.shared : p.routed;
  const long long row = 2LL * f * e + i;
  const uint16_t* x = p.x + t * p.ldx;
  const float g = dot<kW8>(w.gate_up, scales(w.gate_up_scale, e, 2 * f, i, p.d), row, p.d, x, p.bf16);
  const float u = dot<kW8>(w.gate_up, scales(w.gate_up_scale, e, 2 * f, f + i, p.d), row + f, p.d, x, p.bf16);
  const float v = gelu16(g, p.gelu) * u * (shared ? 1.f : p.gates[pair]);
  uint16_t* a = shared ? p.a + static_cast<long long>(pairs) * p.f + static_cast<long long>(t) * f : p.a + static_cast<long long>(pair) * f;
  if ((threadIdx.x & 31) == 0) a[i] = p.bf16 ? float_to_bf16_bits(v) : __half_as_ushort(__float2half_rn(v));
}

template <bool kW8>
__global__ void __launch_bounds__(256) k_layer_down(LayerParams p) {
  const int t = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= p.d) return;
  float sum = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int e = p.ids[t * p.k + j];
    if (e < 0 || e >= p.E) continue;
    sum += dot<kW8>(p.routed.down, scales(p.routed.down_scale, e, p.d, i, p.f), static_cast<long long>(e) * p.d + i, p.f,
                    p.a + static_cast<long long>(t * p.k + j) * p.f, p.bf16);
  }
  if (p.fs)
    sum += dot<kW8>(p.shared.down, scales(p.shared.down_scale, 0, p.d, i, p.fs), i, p.fs,
                    p.a + static_cast<long long>(p.t) * p.k * p.f + static_cast<long long>(t) * p.fs, p.bf16);
  if ((threadIdx.x & 31) != 0) return;
  if (p.out_f32)
    static_cast<float*>(p.y)[t * p.ldy + i] = sum;
  else
    static_cast<uint16_t*>(p.y)[t * p.ldy + i] = p.bf16 ? float_to_bf16_bits(sum) : __half_as_ushort(__float2half_rn(sum));
}

}  // namespace

bool launch_layer(bool weights8, const LayerParams& p, cudaStream_t s) {
  const dim3 up((std::max(p.f, p.fs) + 7) / 8, p.t * p.k + (p.fs ? p.t : 0)), down((p.d + 7) / 8, p.t);
  if (weights8) {
    k_layer_up<true><<<up, 256, 0, s>>>(p);
    k_layer_down<true><<<down, 256, 0, s>>>(p);
  } else {
    k_layer_up<false><<<up, 256, 0, s>>>(p);
    k_layer_down<false><<<down, 256, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess;
}

}  // namespace moe
