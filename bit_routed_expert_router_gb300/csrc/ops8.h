// Launch interface of the norm (norm.cu), of the 8-bit grouped products
// (grouped_mm8.cu) and of the layer for a few tokens (token_layer.cu).  All
// arguments are checked by the C entry points in ops8_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "grouped.h"

namespace moe {

constexpr int kNormMaxD = 16384;
constexpr int kNormParts = 512;   // most rows of partial weight gradients

struct NormParams {
  const void* h = nullptr;
  const void* delta = nullptr;
  const void* weight = nullptr;
  void* h_out = nullptr;
  void* y = nullptr;
  uint8_t* y8 = nullptr;
  float* scale = nullptr;   // [m][ceil(d / 128)]
  long long ldh = 0, ldd = 0, ldo = 0, ldy = 0, ldy8 = 0;   // elements
  int m = 0, d = 0;
  float eps = 0.f, over_d = 0.f;   // over_d: 1 / d, set by the launches
};

struct NormGradParams {
  const void* h = nullptr;
  const void* dy = nullptr;
  const void* dres = nullptr;
  const void* weight = nullptr;
  void* dh = nullptr;
  float* part = nullptr;      // [parts][d], null: no weight gradient
  float* dweight = nullptr;
  long long ldh = 0, lddy = 0, lddres = 0, lddh = 0;
  int m = 0, d = 0, parts = 0;
  float eps = 0.f, over_d = 0.f;   // parts and over_d (1 / d): set by the launches
};

// false: a CUDA call failed.
bool launch_norm(bool bf16, bool delta_f32, const NormParams& p, cudaStream_t s);
bool launch_norm_grad(bool bf16, const NormGradParams& p, cudaStream_t s);

// One grouped product of e4m3 rows and weights [E][n][k], with scales for 128
// values of a row and for 128 x 128 blocks of an expert's weights.
struct Mm8Params {
  const uint8_t* x = nullptr;
  long long ldx = 0;
  const float* sx = nullptr;          // [m][ceil(k / 128)]
  const int32_t* offsets = nullptr;   // [E + 1]
  const uint8_t* w = nullptr;
  const float* sw = nullptr;          // [E][ceil(n / 128)][ceil(k / 128)]
  int E = 1, m = 0, n = 0, k = 0;
  void* y = nullptr;                  // [m][ldy] of `out` (MOE_BF16, ...); gated: e4m3 of n / 2 features
  long long ldy = 0;
  int out = 0;
  float* sa = nullptr;                // gated: [m][ceil(n / 2 / 128)]
  int gelu = 0;
  int limit = 0, stall = 0;           // set by the launches: bounded waits, in 1024 cycles; loads after which they stop
  GaveUp* gave_up = nullptr;          // the same
};

// false: a CUDA call failed.
bool launch_grouped8(bool gated, const Mm8Params& p, cudaStream_t s);

constexpr int kLayerTokens = 32, kLayerTopK = 32;

// A feed-forward network's weights: [2 f][d] and [d][f] (routed: of each expert), of the call's type or e4m3 with the
// scales of 128 x 128 blocks.
struct FfnWeights {
  const void* gate_up = nullptr;
  const void* down = nullptr;
  const float* gate_up_scale = nullptr;
  const float* down_scale = nullptr;
};

struct LayerParams {
  const uint16_t* x = nullptr;
  long long ldx = 0;
  const int32_t* ids = nullptr;     // [t][k]
  const float* gates = nullptr;     // [t][k]
  int t = 0, k = 0, E = 0, d = 0, f = 0, fs = 0;   // fs = 0: no shared expert
  FfnWeights routed, shared;
  uint16_t* a = nullptr;            // workspace: gated products, [t k][f] then [t][fs]
  void* y = nullptr;
  long long ldy = 0;
  int bf16 = 0, out_f32 = 0, gelu = 0;
  int limit = 0, stall = 0;         // set by the launches: bounded waits, in 1024 cycles; loads after which they stop
  GaveUp* gave_up = nullptr;        // the same
};

// false: a CUDA call failed.
bool launch_layer(bool weights8, const LayerParams& p, cudaStream_t s);

}  // namespace moe
