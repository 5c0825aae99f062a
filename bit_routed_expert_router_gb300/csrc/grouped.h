// Launch interface of the 16-bit grouped products (grouped_mm.cu) and of the
// kernels around them (gated_lora.cu).  All arguments are checked by the C
// entry points in ops_api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

enum GmMode { GM_FWD = 0, GM_DGRAD = 1, GM_WGRAD = 2 };
enum GmEpi { GM_PLAIN = 0, GM_GATED = 1, GM_ADAPT = 2, GM_F32 = 3 };   // GM_F32: GM_PLAIN with fp32 outputs

// One grouped product.  "Features" are the output's contiguous dimension,
// "columns" its rows: the grouped rows themselves (GM_FWD, GM_DGRAD), or the n
// rows of each expert's weight gradient (GM_WGRAD, where the grouped rows are
// the reduction).
struct GmParams {
  const int32_t* offsets = nullptr;   // [E + 1] row ranges of the experts; null: one group of all m rows
  int E = 1, m = 0;
  int feat = 0;                       // features (GM_GATED: of a, half the weight rows)
  int red = 0;                        // reduction length (GM_FWD, GM_DGRAD)
  int cols = 0;                       // GM_WGRAD: n
  void* y = nullptr;
  long long ldy = 0;                  // elements
  int out_f32 = 0, bf16 = 0;
  void* h = nullptr;                  // GM_GATED: null or [m][2 feat]
  long long ldh = 0;
  int gelu = 0;
  const int32_t* ids = nullptr;       // GM_ADAPT: adapter of each row
  const uint16_t* b = nullptr;        // [n_adapters][feat][rank]
  const float* u = nullptr;           // [m][rank]: s A x, 32-byte aligned
  int rank = 0, n_adapters = 0;
  int limit = 0, stall = 0;           // set by the launches, see grouped_test_cycles
};

// x: rows [m][ldx]; w: [E][n][k] contiguous (GM_FWD: n features, k reduction;
// GM_DGRAD the reverse; GM_GATED n = 2 feat).  GM_WGRAD: x and dy rows.
struct GmOperands {
  const void* x = nullptr;
  long long ldx = 0;
  const void* w = nullptr;            // or dy for GM_WGRAD
  long long ldw = 0;                  // GM_WGRAD: elements between rows of dy
  int n = 0, k = 0;
};

// false: a CUDA call failed.
bool launch_grouped(int mode, int epi, const GmOperands& o, const GmParams& p, cudaStream_t s);
// Tests: the bounded waits of launches from now on give up after `cycles`, and
// their loading threads stop after `loads` (0 or less: the default of either,
// about two seconds and never).
void grouped_test_cycles(int64_t cycles);
void grouped_test_loads(int64_t loads);
// Synchronises the stream; news: a wait ran out on the current device since the
// last call with this stream.
bool grouped_gave_up(cudaStream_t s, bool* news);

bool launch_gated_grad(bool bf16, int gelu, const void* h, long long ldh, const void* da, long long ldda, void* dh,
                       long long lddh, int m, int f, const int32_t* n_rows, cudaStream_t s);

// u[t] = scale[id] A[id] x[t] for every row with an adapter: few rows, and many
// (o.x, o.w = A; p: m, red, rank, n_adapters, ids, bf16).
bool launch_adapter_down_many(const GmOperands& o, const GmParams& p, const float* scale, float* u, cudaStream_t s);
bool launch_adapter_down(bool bf16, const void* x, long long ldx, int t, const void* a, const float* scale,
                         const int32_t* ids, int n_adapters, int rank, int k, float* u, cudaStream_t s);

}  // namespace moe
