// A routed layer and its shared expert for up to 32 tokens, in two kernels:
//
//   up     a[i] = gate GELU(g) u,  [g, u] = Wgu[e] x[t]     for the tokens of each picked expert, rounded to the call's type
//   down   y[t] = sum_e Wd[e] a[e, t]                       over the experts that t names, and the shared one
//
// The weights of the picked experts are read once and nothing else is of any
// size, so both kernels stream them: one warp copies chunks of 16 weight rows,
// and of the token rows that go with them, into a ring of stages (cp.async.bulk,
// one copy a row), eight warps share the 32- or 64-value steps of a chunk and
// multiply them as m16n8k16 fragments, weights on the M side.  A lane reads 16
// bytes of a row at a time: the order of k within a step is the same in both
// operands, which is all that a product needs.  e4m3 weights become 16-bit ones
// in registers (exact); each block of 128 is summed by itself, then scaled.
//
// up: a unit is 8 features: their 8 gate and 8 up rows are the 16 rows, so that a
// lane ends with both factors of its values.  Columns: the expert's tokens.
// down: a unit is 16 outputs over all picked experts, its chunks dealt out to a
// cluster's CTAs, which add their sums through distributed shared memory in rank
// order.  Columns: all tokens; an expert's sums are added to those that name it
// only, so that weights that are not finite stay with their own tokens.  The
// kernel starts while the first one runs and fills its ring with weights.
#include <algorithm>

#include "gelu16.cuh"
#include "grouped.h"
#include "ops8.h"
#include "quant8.cuh"
#include "waits.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);
constexpr int kChunkBytes = 1024;   // of a weight row, at most
constexpr int kMaxStages = 8;
constexpr int kBudget = 72 * 1024;  // shared memory of a CTA: three fit an SM, so that the down kernel's ring fills early

struct Slot {
  int expert;      // -1: the shared expert
  uint32_t mask;   // its tokens
  int base;        // its rows of a (the shared one's: in its own part)
};

// Host and device: what a launch's CTA keeps, and where.
struct Plan {
  int kc_d, kc_f, kc_fs;      // values of a chunk: along d, f and f_shared
  int pitch_w, pitch_x;       // bytes between staged rows: weights, tokens
  int stage, stages;
  int slots;                  // most picked experts
  int at_red, at_mask, at_ids, at_gates, at_slots, bytes;
};

__host__ __device__ __forceinline__ int divide_up(int a, int b) { return (a + b - 1) / b; }

// Equal chunks of at most kChunkBytes, whole steps each.
int chunk_of(int k, bool w8) {
  const int most = w8 ? kChunkBytes : kChunkBytes / 2, unit = w8 ? 128 : 32;
  return k == 0 ? 0 : divide_up(divide_up(k, divide_up(k, most)), unit) * unit;
}

struct Chunk {
  int slot;            // index, n_slots for the shared expert
  int k0, k;           // first value and length
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <bool kBf16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 values in the call's type (exact in both).
template <bool kBf16>
__device__ __forceinline__ uint32_t widen8(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  if (!kBf16) return h;
  const __nv_bfloat162 b = __floats2bfloat162_rn(half_lo(h), half_hi(h));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// c += 16 weight rows times up to 8 kNt token rows over this warp's steps of a staged chunk.  w: the stage; xr[j]: this
// lane's token row of columns 8 j .., 0 for none.  With e4m3 weights the chunk is one block a warp, and c is scaled later.
template <bool kBf16, bool kW8, int kNt>
__device__ __forceinline__ void multiply(float (&c)[kNt][4], uint32_t w, const uint32_t (&xr)[kNt], int n_cols, int pitch_w,
                                         int k, int warp, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (kW8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 128 * warp + 64 * h;
      if (at >= k) return;
      const bool in = at + 16 * t < k;
      const uint4 w0 = in ? lds16(w + g * pitch_w + at + 16 * t) : zero, w1 = in ? lds16(w + (g + 8) * pitch_w + at + 16 * t) : zero;
      const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
      uint32_t a[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i][0] = widen8<kBf16>(lo[i]), a[i][1] = widen8<kBf16>(hi[i]), a[i][2] = widen8<kBf16>(lo[i] >> 16),
        a[i][3] = widen8<kBf16>(hi[i] >> 16);
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
        if (8 * j >= n_cols) break;
        const bool on = in && xr[j];
        const uint4 x0 = on ? lds16(xr[j] + 2 * at + 32 * t) : zero, x1 = on ? lds16(xr[j] + 2 * at + 32 * t + 16) : zero;
        mma16<kBf16>(c[j], a[0][0], a[0][1], a[0][2], a[0][3], x0.x, x0.y);
        mma16<kBf16>(c[j], a[1][0], a[1][1], a[1][2], a[1][3], x0.z, x0.w);
        mma16<kBf16>(c[j], a[2][0], a[2][1], a[2][2], a[2][3], x1.x, x1.y);
        mma16<kBf16>(c[j], a[3][0], a[3][1], a[3][2], a[3][3], x1.z, x1.w);
      }
    }
  } else {
    for (int at = 32 * warp; at < k; at += 32 * kWarps) {
      const bool in = at + 8 * t < k;
      const uint32_t off = 2 * at + 16 * t;
      const uint4 w0 = in ? lds16(w + g * pitch_w + off) : zero, w1 = in ? lds16(w + (g + 8) * pitch_w + off) : zero;
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
        if (8 * j >= n_cols) break;
        const uint4 x = in && xr[j] ? lds16(xr[j] + off) : zero;
        mma16<kBf16>(c[j], w0.x, w1.x, w0.y, w1.y, x.x, x.y);
        mma16<kBf16>(c[j], w0.z, w1.z, w0.w, w1.w, x.z, x.w);
      }
    }
  }
}

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  Waits waits;
  int n_slots;
};

// The picked experts in order, each with its tokens; every thread of the CTA.
__device__ void list_slots(const LayerParams& p, const Plan& P, uint8_t* smem, Shared& S) {
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + P.at_mask);
  int* ids = reinterpret_cast<int*>(smem + P.at_ids);
  float* gates = reinterpret_cast<float*>(smem + P.at_gates);
  Slot* slots = reinterpret_cast<Slot*>(smem + P.at_slots);
  for (int i = threadIdx.x; i < p.E; i += kThreads) mask[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.t * p.k; i += kThreads) {
    const int e = __ldcg(p.ids + i);
    ids[i] = e;
    gates[i] = __ldcg(p.gates + i);
    if (e >= 0 && e < p.E) atomicOr(&mask[e], 1u << (i / p.k));
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const uint32_t m = e0 + lane < p.E ? mask[e0 + lane] : 0;
      const uint32_t picked = __ballot_sync(0xFFFFFFFFu, m != 0), before = picked & ((1u << lane) - 1);
      int sum = __popc(m);
      const int own = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      if (m) slots[n + __popc(before)] = {e0 + lane, m, rows + sum - own};
      n += __popc(picked);
      rows += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) {
      S.n_slots = n;
      slots[n] = {-1, p.t == 32 ? 0xFFFFFFFFu : (1u << p.t) - 1, 0};
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void init_ring(Shared& S, const LayerParams& p, int stages) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], kWarps);
    }
    S.waits.abort = 0;
    S.waits.limit = p.limit;
    fence_mbar_init();
  }
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (; n > 0; --n) m &= m - 1;
  return __ffs(m) - 1;
}

// ------------------------------------------------------------------ up

template <bool kBf16, bool kW8, int kNt>
__global__ void __launch_bounds__(kThreads) k_layer_up(const __grid_constant__ LayerParams p, const __grid_constant__ Plan P) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  init_ring(S, p, P.stages);
  pdl_wait();
  pdl_trigger();
  list_slots(p, P, smem, S);
  const Slot* slots = reinterpret_cast<const Slot*>(smem + P.at_slots);
  const int n_slots = S.n_slots, per = p.f / 8, routed = n_slots * per, units = routed + p.fs / 8;
  const int chunks = divide_up(p.d, P.kc_d);
  constexpr int kSize = kW8 ? 1 : 2;   // bytes of a weight

  if (warp == kWarps) {
    int it = 0;
    bool go = true;
    for (int unit = blockIdx.x; go && unit < units; unit += gridDim.x) {
      const bool shared = unit >= routed;
      const Slot sl = slots[shared ? n_slots : unit / per];
      const int f = shared ? p.fs : p.f, f0 = 8 * (shared ? unit - routed : unit % per), rows = __popc(sl.mask);
      const uint8_t* w = static_cast<const uint8_t*>(shared ? p.shared.gate_up : p.routed.gate_up) +
                         ((shared ? 0LL : 2LL * f * sl.expert) + f0) * p.d * kSize;
      // lane l copies weight row l (gate, then up) or token row l - 16, and l + 16
      const uint8_t* from_w = w + (lane < 8 ? lane : lane - 8 + static_cast<long long>(f)) * p.d * kSize;
      const int t0 = lane >= 16 && lane - 16 < rows ? nth_bit(sl.mask, lane - 16) : -1;
      const int t1 = lane >= 16 && lane < rows ? nth_bit(sl.mask, lane) : -1;
      for (int c = 0; c < chunks; ++c, ++it) {
        const int s = it % P.stages, k0 = c * P.kc_d, k = min(P.kc_d, p.d - k0);
        if (!(go = it < p.stall && wait_bar_warp(&S.empty[s], ((it / P.stages) & 1) ^ 1, &S.waits))) break;
        uint8_t* at = smem + s * P.stage;
        if (lane == 0) mbar_arrive_expect_tx(&S.full[s], 16 * k * kSize + rows * k * 2);
        __syncwarp();
        if (lane < 16) {
          bulk_g2s(at + lane * P.pitch_w, from_w + static_cast<long long>(k0) * kSize, k * kSize, &S.full[s]);
        } else {
          uint8_t* x = at + 16 * P.pitch_w;
          if (t0 >= 0) bulk_g2s(x + (lane - 16) * P.pitch_x, p.x + t0 * p.ldx + k0, 2 * k, &S.full[s]);
          if (t1 >= 0) bulk_g2s(x + lane * P.pitch_x, p.x + t1 * p.ldx + k0, 2 * k, &S.full[s]);
        }
      }
    }
  } else {
    const int g = lane >> 2;
    int it = 0, turn = 0;
    bool ok = true;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x, turn ^= 1) {
      const bool shared = unit >= routed;
      const Slot sl = slots[shared ? n_slots : unit / per];
      const int f = shared ? p.fs : p.f, f0 = 8 * (shared ? unit - routed : unit % per), rows = __popc(sl.mask);
      const float* scale = nullptr;
      int up_scale = 0;
      if (kW8) {
        const int kb = divide_up(p.d, 128);
        scale = (shared ? p.shared.gate_up_scale : p.routed.gate_up_scale + static_cast<long long>(sl.expert) * divide_up(2 * f, 128) * kb) +
                f0 / 128 * kb;
        up_scale = ((f + f0) / 128 - f0 / 128) * kb;
      }
      float acc[kNt][4] = {};
      for (int c = 0; c < chunks; ++c, ++it) {
        const int s = it % P.stages, k0 = c * P.kc_d, k = min(P.kc_d, p.d - k0);
        float sg = 0.f, su = 0.f;
        if (kW8 && 128 * warp < k) sg = __ldg(scale + k0 / 128 + warp), su = __ldg(scale + up_scale + k0 / 128 + warp);
        ok = ok && wait_bar_warp(&S.full[s], (it / P.stages) & 1, &S.waits);
        if (ok) {
          const uint32_t w = smem_u32(smem + s * P.stage), x = w + 16 * P.pitch_w;
          uint32_t xr[kNt];
#pragma unroll
          for (int j = 0; j < kNt; ++j) xr[j] = 8 * j + g < rows ? x + (8 * j + g) * P.pitch_x : 0;
          if (kW8) {
            float block[kNt][4] = {};
            multiply<kBf16, kW8, kNt>(block, w, xr, rows, P.pitch_w, k, warp, lane);
#pragma unroll
            for (int j = 0; j < kNt; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (128 * warp < k) acc[j][i] = fmaf(block[j][i], i < 2 ? sg : su, acc[j][i]);
          } else {
            multiply<kBf16, kW8, kNt>(acc, w, xr, rows, P.pitch_w, k, warp, lane);
          }
        }
        __syncwarp();
        if (lane == 0) mbarrier_arrive(&S.empty[s]);
      }
      // the warps' sums in turn: 8 features x 8 kNt columns, both factors
      float4* red = reinterpret_cast<float4*>(smem + P.at_red) + turn * kWarps * kNt * 32;
#pragma unroll
      for (int j = 0; j < kNt; ++j) red[(warp * kNt + j) * 32 + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      consumers_sync();
      const int i = tid & 7, col = tid >> 3;   // feature, column
      if (ok && col < rows && col < 8 * kNt) {
        const float* from = reinterpret_cast<const float*>(red + (col >> 3) * 32 + 4 * i + ((col & 7) >> 1)) + (col & 1);
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) gate += from[v * kNt * 128], up += from[v * kNt * 128 + 2];
        float weight = 1.f;
        if (!shared) {
          const int* ids = reinterpret_cast<const int*>(smem + P.at_ids);
          const float* gates = reinterpret_cast<const float*>(smem + P.at_gates);
          const int t = nth_bit(sl.mask, col);
          weight = 0.f;
          for (int j = 0; j < p.k; ++j) weight += ids[t * p.k + j] == sl.expert ? gates[t * p.k + j] : 0.f;
        }
        const float v = weight * (gelu16(gate, p.gelu) * up);
        uint16_t* a = p.a + (shared ? static_cast<long long>(p.t) * p.k * p.f : 0LL) + static_cast<long long>(sl.base + col) * f + f0 + i;
        *a = kBf16 ? float_to_bf16_bits(v) : __half_as_ushort(__float2half_rn(v));
      }
    }
  }
  __syncthreads();
  if (S.waits.abort) report_and_settle();
}

// ------------------------------------------------------------------ down

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float ld_rank(const float* at, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// The chunks of a unit: each picked expert's along f, then the shared expert's.
struct DownChunks {
  int n_slots, per, all, f, fs, kc, kcs;
  __device__ __forceinline__ Chunk at(int i) const {
    Chunk c;
    c.slot = min(i / per, n_slots);
    const int first = i - c.slot * per;
    const bool shared = c.slot == n_slots;
    c.k0 = first * (shared ? kcs : kc);
    c.k = min(shared ? kcs : kc, (shared ? fs : f) - c.k0);
    return c;
  }
};

template <bool kBf16, bool kW8, int kNt>
__global__ void __launch_bounds__(kThreads) k_layer_down(const __grid_constant__ LayerParams p, const __grid_constant__ Plan P,
                                                         int split) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), d0 = blockIdx.x / split * 16;
  constexpr int kSize = kW8 ? 1 : 2;
  init_ring(S, p, P.stages);
  // ids and weights are older than the first kernel, which let this one start after its own wait
  list_slots(p, P, smem, S);
  const Slot* slots = reinterpret_cast<const Slot*>(smem + P.at_slots);
  DownChunks C;
  C.n_slots = S.n_slots, C.f = p.f, C.fs = p.fs, C.kc = P.kc_f, C.kcs = P.kc_fs, C.per = divide_up(p.f, P.kc_f);
  C.all = C.n_slots * C.per + (p.fs ? divide_up(p.fs, P.kc_fs) : 0);
  const int first = static_cast<int>(static_cast<long long>(C.all) * rank / split);
  const int n = static_cast<int>(static_cast<long long>(C.all) * (rank + 1) / split) - first;

  if (warp == kWarps) {
    const auto rows_of = [&](const Chunk& c) { return __popc(slots[c.slot].mask); };
    const auto load_w = [&](int i, const Chunk& c, int s) {
      const bool shared = c.slot == C.n_slots;
      const int f = shared ? p.fs : p.f;
      if (lane == 0) mbar_arrive_expect_tx(&S.full[s], 16 * c.k * kSize + rows_of(c) * c.k * 2);
      __syncwarp();
      const uint8_t* w = static_cast<const uint8_t*>(shared ? p.shared.down : p.routed.down) +
                         (((shared ? 0LL : static_cast<long long>(slots[c.slot].expert) * p.d) + d0 + lane) * f + c.k0) * kSize;
      if (lane < 16) bulk_g2s(smem + s * P.stage + lane * P.pitch_w, w, c.k * kSize, &S.full[s]);
    };
    const auto load_a = [&](const Chunk& c, int s) {
      const bool shared = c.slot == C.n_slots;
      const int f = shared ? p.fs : p.f;
      const uint16_t* a = p.a + (shared ? static_cast<long long>(p.t) * p.k * p.f : 0LL) +
                          static_cast<long long>(slots[c.slot].base + lane) * f + c.k0;
      if (lane < rows_of(c)) bulk_g2s(smem + s * P.stage + 16 * P.pitch_w + lane * P.pitch_x, a, 2 * c.k, &S.full[s]);
    };
    const int early = min(min(n, P.stages), p.stall);
    for (int i = 0; i < early; ++i) load_w(i, C.at(first + i), i);
    pdl_wait();
    for (int i = 0; i < early; ++i) load_a(C.at(first + i), i);
    for (int i = early; i < min(n, p.stall); ++i) {
      const int s = i % P.stages;
      if (!wait_bar_warp(&S.empty[s], ((i / P.stages) & 1) ^ 1, &S.waits)) break;
      const Chunk c = C.at(first + i);
      load_w(i, c, s);
      load_a(c, s);
    }
  }
  pdl_wait();   // y may be in use until here
  pdl_trigger();
  float* part = reinterpret_cast<float*>(smem + P.at_red);   // [column][16] of this CTA, behind the warps' sums
  constexpr int kRed = kWarps * kNt * 32 * 4;
  bool ok = true;
  if (warp < kWarps) {
    const int g = lane >> 2, t = lane & 3;
    float acc[kNt][4] = {}, own[kNt][4] = {};   // of all experts, of the one at hand
    const int kb = divide_up(p.f, 128), kbs = divide_up(p.fs, 128), db = divide_up(p.d, 128);
    for (int i = 0; i < n; ++i) {
      const int s = i % P.stages;
      const Chunk c = C.at(first + i);
      const uint32_t mask = slots[c.slot].mask;
      float sc = 0.f;
      if (kW8 && 128 * warp < c.k)
        sc = c.slot == C.n_slots
                 ? __ldg(p.shared.down_scale + d0 / 128 * kbs + c.k0 / 128 + warp)
                 : __ldg(p.routed.down_scale + (static_cast<long long>(slots[c.slot].expert) * db + d0 / 128) * kb + c.k0 / 128 + warp);
      ok = ok && wait_bar_warp(&S.full[s], (i / P.stages) & 1, &S.waits);
      if (ok) {
        const uint32_t w = smem_u32(smem + s * P.stage), x = w + 16 * P.pitch_w;
        uint32_t xr[kNt];
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
          const int col = 8 * j + g;
          xr[j] = (mask >> col) & 1 ? x + __popc(mask & ((1u << col) - 1)) * P.pitch_x : 0;
        }
        if (kW8) {
          float block[kNt][4] = {};
          multiply<kBf16, kW8, kNt>(block, w, xr, 32, P.pitch_w, c.k, warp, lane);
#pragma unroll
          for (int j = 0; j < kNt; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (128 * warp < c.k) own[j][v] = fmaf(block[j][v], sc, own[j][v]);
        } else {
          multiply<kBf16, kW8, kNt>(own, w, xr, 32, P.pitch_w, c.k, warp, lane);
        }
        if (i + 1 == n || C.at(first + i + 1).slot != c.slot) {
#pragma unroll
          for (int j = 0; j < kNt; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              if ((mask >> (8 * j + 2 * t + (v & 1))) & 1) acc[j][v] += own[j][v];
              own[j][v] = 0.f;
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbarrier_arrive(&S.empty[s]);
    }
    float4* red = reinterpret_cast<float4*>(smem + P.at_red);
#pragma unroll
    for (int j = 0; j < kNt; ++j) red[(warp * kNt + j) * 32 + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    consumers_sync();
    const int row = tid & 15;
    for (int col = tid >> 4; col < p.t; col += 16) {
      const float* from = part + ((col >> 3) * 32 + 4 * (row & 7) + ((col & 7) >> 1)) * 4 + (col & 1) + (row >> 3) * 2;
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += from[v * kNt * 128];
      part[kRed + col * 16 + row] = sum;
    }
  }
  ok = ok && !S.waits.abort;
  if (split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (ok)
    for (int i = tid; i < 16 * p.t; i += kThreads) {
      const int col = i >> 4, row = i & 15;
      if (col % split != rank) continue;
      float sum = 0.f;
      if (split == 1)
        sum = part[kRed + i];
      else
        for (int r = 0; r < split; ++r) sum += ld_rank(part + kRed + i, r);
      const long long at = col * p.ldy + d0 + row;
      if (p.out_f32)
        static_cast<float*>(p.y)[at] = sum;
      else
        static_cast<uint16_t*>(p.y)[at] = kBf16 ? float_to_bf16_bits(sum) : __half_as_ushort(__float2half_rn(sum));
    }
  if (split > 1) cluster_sync();   // the others may still read this CTA's sums
  __syncthreads();
  if (S.waits.abort) report_and_settle();
}

// ------------------------------------------------------------------ launches

int padded(int bytes, int to) { return (bytes + 127) / 128 * 128 + to; }

// e4m3 rows have half the bytes of the token rows beside them, which two words a lane of 32 bytes apart read: 16 bytes more
// than a multiple of 128 keep eight lanes apart there, 64 where a row's four lanes read 64 bytes.
Plan make_plan(const LayerParams& p, bool w8, bool down) {
  Plan P{};
  P.kc_d = chunk_of(p.d, w8), P.kc_f = chunk_of(p.f, w8), P.kc_fs = chunk_of(p.fs, w8);
  const int kc = down ? std::max(P.kc_f, P.kc_fs) : P.kc_d, nt = p.t <= 8 ? 1 : 4;
  P.pitch_w = padded(kc * (w8 ? 1 : 2), 64), P.pitch_x = padded(2 * kc, w8 ? 16 : 64);
  P.stage = (16 * P.pitch_w + p.t * P.pitch_x + 127) / 128 * 128;
  P.slots = std::min(p.t * p.k, p.E);
  const int red = kWarps * nt * 512 * (down ? 1 : 2) + (down ? nt * 512 : 0);
  const int lists = 4 * p.E + 8 * p.t * p.k + static_cast<int>(sizeof(Slot)) * (P.slots + 1) + 64;
  const int most = down ? kMaxStages : kMaxStages;
  P.stages = std::clamp((kBudget - red - lists) / P.stage, 2, most);
  P.at_red = P.stages * P.stage;
  P.at_mask = P.at_red + red;
  P.at_ids = P.at_mask + 4 * p.E;
  P.at_gates = P.at_ids + 4 * p.t * p.k;
  P.at_slots = P.at_gates + 4 * p.t * p.k;
  P.bytes = P.at_slots + static_cast<int>(sizeof(Slot)) * (P.slots + 1);
  return P;
}

template <typename K, typename... A>
bool launch(K kernel, int grid, const Plan& P, int cluster, cudaStream_t s, const A&... args) {
  if (P.bytes > 48 * 1024 - 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P.bytes) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = P.bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <bool kBf16, bool kW8, int kNt>
bool launch_both(const LayerParams& p, int sms, cudaStream_t s) {
  const Plan up = make_plan(p, kW8, false), down = make_plan(p, kW8, true);
  // every CTA the same number of units, as far as the picked experts are known here: two CTAs an SM
  const int units = up.slots * (p.f / 8) + p.fs / 8, rounds = divide_up(units, 2 * sms);
  if (!launch(k_layer_up<kBf16, kW8, kNt>, divide_up(units, rounds), up, 1, s, p, up)) return false;
  const int blocks = p.d / 16, chunks = down.slots * divide_up(p.f, down.kc_f) + (p.fs ? divide_up(p.fs, down.kc_fs) : 0);
  int split = 1;
  while (split < 8 && 2 * split * blocks <= 2 * sms && 2 * split <= chunks) split *= 2;
  return launch(k_layer_down<kBf16, kW8, kNt>, blocks * split, down, split, s, p, down, split);
}

template <bool kBf16, bool kW8>
bool launch_of(const LayerParams& p, int sms, cudaStream_t s) {
  return p.t <= 8 ? launch_both<kBf16, kW8, 1>(p, sms, s) : launch_both<kBf16, kW8, 4>(p, sms, s);
}

}  // namespace

bool launch_layer(bool weights8, const LayerParams& params, cudaStream_t s) {
  LayerParams p = params;
  const WaitLimits l = wait_limits();
  p.limit = l.cycles1024, p.stall = l.loads;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return false;
  if (weights8) return p.bf16 ? launch_of<true, true>(p, sms, s) : launch_of<false, true>(p, sms, s);
  return p.bf16 ? launch_of<true, false>(p, sms, s) : launch_of<false, false>(p, sms, s);
}

bool layer_gave_up(cudaStream_t s, uint32_t* count) {
  return cudaMemcpyFromSymbolAsync(count, g_gave_up, sizeof(*count), 0, cudaMemcpyDeviceToHost, s) == cudaSuccess;
}

}  // namespace moe
