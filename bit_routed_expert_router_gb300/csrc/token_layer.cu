// A routed layer and its shared expert for up to 32 tokens, in two kernels:
//
//   up     a[i] = gate GELU(g) u,  [g, u] = Wgu[e] x[t]     for the tokens of each picked expert, rounded to the call's type
//   down   y[t] = sum_e Wd[e] a[e, t]                       over the experts that t names, and the shared one
//
// The weights of the picked experts are read once and nothing else is of any
// size, so both kernels stream them: one thread copies chunks of 16 weight rows
// (one TMA load: a bulk copy a row took about 85 cycles each, 52 us for one token
// where the weights take 21), and of the token rows that go with them, into a ring
// of stages; eight warps share a chunk's steps of 64 bytes and multiply them as
// m16n8k16 fragments, weights on the M side.  A lane reads 16 bytes of a row at a
// time: the order of k within a step is the same in both operands, which is all
// that a product needs, and chunks of an odd number of steps keep the rows of eight
// lanes in different banks.  e4m3 weights become 16-bit ones in registers (exact);
// each step's sums are scaled by themselves.
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
#include "tensor_map.h"
#include "waits.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);
constexpr int kStep = 64, kChunkBytes = 15 * kStep;   // of a weight row; a chunk at most
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
  int pitch_x;                // bytes between staged token rows
  int stage, stages;
  int slots;                  // most picked experts
  int at_red, at_mask, at_ids, at_gates, at_slots, bytes;
};

__host__ __device__ __forceinline__ int divide_up(int a, int b) { return (a + b - 1) / b; }

// Equal chunks of an odd number of steps, in values.
int chunk_of(int k, int size) {
  if (k == 0) return 0;
  const int chunks = divide_up(k * size, kChunkBytes), steps = divide_up(divide_up(k * size, chunks), kStep);
  return (steps | 1) * kStep / size;
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

// c += 16 weight rows times up to 8 kNt token rows over one step of a staged chunk, which ends (k values) in it or behind it.
// xr[j]: this lane's token row of columns 8 j .., 0 for none.
template <bool kBf16, bool kW8, int kNt>
__device__ __forceinline__ void multiply(float (&c)[kNt][4], uint32_t w, int pitch_w, const uint32_t (&xr)[kNt], int n_cols, int at,
                                         int k, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint32_t from = w + g * pitch_w + (kW8 ? at : 2 * at) + 16 * t;
  const uint4 w0 = lds16(from), w1 = lds16(from + 8 * pitch_w);   // zeros past k
  if (kW8) {
    const bool in = at + 16 * t < k;
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
  } else {
    const bool in = at + 8 * t < k;
#pragma unroll
    for (int j = 0; j < kNt; ++j) {
      if (8 * j >= n_cols) break;
      const uint4 x = in && xr[j] ? lds16(xr[j] + 2 * at + 16 * t) : zero;
      mma16<kBf16>(c[j], w0.x, w1.x, w0.y, w1.y, x.x, x.y);
      mma16<kBf16>(c[j], w0.z, w1.z, w0.w, w1.w, x.z, x.w);
    }
  }
}

// This warp's steps of a staged chunk of kc values, of which k are there; with e4m3 weights scaled by lo[block of 128] (rows
// 0 .. 7) and hi[block] (8 .. 15), blocks counted from k0.
template <bool kBf16, bool kW8, int kNt>
__device__ __forceinline__ void chunk_products(float (&acc)[kNt][4], uint32_t w, const uint32_t (&xr)[kNt], int n_cols, int kc,
                                               int k, int k0, const float* lo, const float* hi, int warp, int lane) {
  constexpr int kValues = kW8 ? kStep : kStep / 2;
  if (kW8) {
    float s[2][2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = kValues * (warp + kWarps * i);
      if (at < k) s[i][0] = __ldg(lo + (k0 + at) / 128), s[i][1] = __ldg(hi + (k0 + at) / 128);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = kValues * (warp + kWarps * i);
      if (at >= k) break;
      float part[kNt][4] = {};
      multiply<kBf16, kW8, kNt>(part, w, kc, xr, n_cols, at, k, lane);
#pragma unroll
      for (int j = 0; j < kNt; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][v] = fmaf(part[j][v], s[i][v >> 1], acc[j][v]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = kValues * (warp + kWarps * i);
      if (at < k) multiply<kBf16, kW8, kNt>(acc, w, 2 * kc, xr, n_cols, at, k, lane);
    }
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// 16 weight rows: [gate, up] x 8 features of an expert, or 16 outputs.
__device__ __forceinline__ void load_up(uint8_t* to, const CUtensorMap* map, int word, int f0, int e, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(smem_u32(to)), "l"(reinterpret_cast<uint64_t>(map)), "r"(word), "r"(f0), "r"(0), "r"(e), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void load_down(uint8_t* to, const CUtensorMap* map, int word, int d0, int e, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(smem_u32(to)), "l"(reinterpret_cast<uint64_t>(map)), "r"(word), "r"(d0), "r"(e), "r"(smem_u32(bar))
      : "memory");
}

// The weights of the routed and of the shared expert, as 32-bit words.
struct Maps {
  CUtensorMap routed, shared;
};

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
__global__ void __launch_bounds__(kThreads) k_layer_up(const __grid_constant__ Maps maps, const __grid_constant__ LayerParams p, const __grid_constant__ Plan P) {
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
    if (elect_one()) {
      int it = 0;
      bool go = true;
      for (int unit = blockIdx.x; go && unit < units; unit += gridDim.x) {
        const bool shared = unit >= routed;
        const Slot sl = slots[shared ? n_slots : unit / per];
        const int f0 = 8 * (shared ? unit - routed : unit % per), rows = __popc(sl.mask);
        for (int c = 0; c < chunks; ++c, ++it) {
          const int s = it % P.stages, k0 = c * P.kc_d, k = min(P.kc_d, p.d - k0);
          if (!(go = it < p.stall && wait_bar(&S.empty[s], ((it / P.stages) & 1) ^ 1, &S.waits))) break;
          uint8_t* at = smem + s * P.stage;
          mbar_arrive_expect_tx(&S.full[s], 16 * P.kc_d * kSize + rows * k * 2);
          load_up(at, shared ? &maps.shared : &maps.routed, k0 * kSize / 4, f0, max(sl.expert, 0), &S.full[s]);
          uint32_t left = sl.mask;
          at += 16 * P.kc_d * kSize;
          for (int i = 0; i < rows; ++i, left &= left - 1, at += P.pitch_x)
            bulk_g2s(at, p.x + (__ffs(left) - 1) * p.ldx + k0, 2 * k, &S.full[s]);
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
        ok = ok && wait_bar_warp(&S.full[s], (it / P.stages) & 1, &S.waits);
        if (ok) {
          const uint32_t w = smem_u32(smem + s * P.stage), x = w + 16 * P.kc_d * kSize;
          uint32_t xr[kNt];
#pragma unroll
          for (int j = 0; j < kNt; ++j) xr[j] = 8 * j + g < rows ? x + (8 * j + g) * P.pitch_x : 0;
          chunk_products<kBf16, kW8, kNt>(acc, w, xr, rows, P.kc_d, k, k0, scale, scale + up_scale, warp, lane);
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
__global__ void __launch_bounds__(kThreads) k_layer_down(const __grid_constant__ Maps maps, const __grid_constant__ LayerParams p,
                                                         const __grid_constant__ Plan P, int split) {
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
    if (elect_one()) {
      const auto load_w = [&](const Chunk& c, int s) {
        const bool shared = c.slot == C.n_slots;
        const int kc = shared ? P.kc_fs : P.kc_f;
        mbar_arrive_expect_tx(&S.full[s], 16 * kc * kSize + __popc(slots[c.slot].mask) * c.k * 2);
        load_down(smem + s * P.stage, shared ? &maps.shared : &maps.routed, c.k0 * kSize / 4, d0, max(slots[c.slot].expert, 0),
                  &S.full[s]);
      };
      const auto load_a = [&](const Chunk& c, int s) {
        const bool shared = c.slot == C.n_slots;
        const int f = shared ? p.fs : p.f, rows = __popc(slots[c.slot].mask);
        const uint16_t* a = p.a + (shared ? static_cast<long long>(p.t) * p.k * p.f : 0LL) +
                            static_cast<long long>(slots[c.slot].base) * f + c.k0;
        uint8_t* to = smem + s * P.stage + 16 * (shared ? P.kc_fs : P.kc_f) * kSize;
        for (int i = 0; i < rows; ++i, a += f, to += P.pitch_x) bulk_g2s(to, a, 2 * c.k, &S.full[s]);
      };
      const int early = min(min(n, P.stages), p.stall);
      for (int i = 0; i < early; ++i) load_w(C.at(first + i), i);
      pdl_wait();
      for (int i = 0; i < early; ++i) load_a(C.at(first + i), i);
      for (int i = early; i < min(n, p.stall); ++i) {
        const int s = i % P.stages;
        if (!wait_bar(&S.empty[s], ((i / P.stages) & 1) ^ 1, &S.waits)) break;
        const Chunk c = C.at(first + i);
        load_w(c, s);
        load_a(c, s);
      }
    }
    __syncwarp();
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
      const bool shared = c.slot == C.n_slots;
      const int kc = shared ? P.kc_fs : P.kc_f;
      const float* scale = !kW8 ? nullptr
                           : shared ? p.shared.down_scale + d0 / 128 * kbs
                                    : p.routed.down_scale + (static_cast<long long>(slots[c.slot].expert) * db + d0 / 128) * kb;
      ok = ok && wait_bar_warp(&S.full[s], (i / P.stages) & 1, &S.waits);
      if (ok) {
        const uint32_t w = smem_u32(smem + s * P.stage), x = w + 16 * kc * kSize;
        uint32_t xr[kNt];
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
          const int col = 8 * j + g;
          xr[j] = (mask >> col) & 1 ? x + __popc(mask & ((1u << col) - 1)) * P.pitch_x : 0;
        }
        chunk_products<kBf16, kW8, kNt>(own, w, xr, 32, kc, c.k, c.k0, scale, scale, warp, lane);
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

// e4m3 rows have half the bytes of the token rows beside them, which two words a lane of 32 bytes apart read: 16 bytes more
// than a multiple of 128 keep eight lanes apart there, 64 where a row's four lanes read 64 bytes.
Plan make_plan(const LayerParams& p, bool w8, bool down) {
  Plan P{};
  const int size = w8 ? 1 : 2;
  P.kc_d = chunk_of(p.d, size), P.kc_f = chunk_of(p.f, size), P.kc_fs = chunk_of(p.fs, size);
  const int kc = down ? std::max(P.kc_f, P.kc_fs) : P.kc_d, nt = p.t <= 8 ? 1 : 4;
  P.pitch_x = divide_up(2 * kc, 128) * 128 + (w8 ? 16 : 64);
  P.stage = divide_up(16 * kc * size + p.t * P.pitch_x, 128) * 128;
  P.slots = std::min(p.t * p.k, p.E);
  const int red = kWarps * nt * 512 * (down ? 1 : 2) + (down ? nt * 512 : 0);
  const int lists = 4 * p.E + 8 * p.t * p.k + static_cast<int>(sizeof(Slot)) * (P.slots + 1) + 64;
  P.stages = std::clamp((kBudget - red - lists) / P.stage, 2, kMaxStages);
  P.at_red = P.stages * P.stage;
  P.at_mask = P.at_red + red;
  P.at_ids = P.at_mask + 4 * p.E;
  P.at_gates = P.at_ids + 4 * p.t * p.k;
  P.at_slots = P.at_gates + 4 * p.t * p.k;
  P.bytes = P.at_slots + static_cast<int>(sizeof(Slot)) * (P.slots + 1);
  return P;
}

bool encode_words(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                  const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dim, stride,
                          box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [E][2][f][d] in boxes of kc values x 8 features x both halves.
bool map_up(CUtensorMap* m, const void* base, int E, int f, int d, int size, int kc) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * size;
  const cuuint64_t dim[4] = {row / 4, static_cast<cuuint64_t>(f), 2, static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[3] = {row, row * f, row * 2 * f};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(kc * size / 4), 8, 2, 1};
  return encode_words(m, base, 4, dim, stride, box);
}

// [E][d][f] in boxes of kc values x 16 outputs.
bool map_down(CUtensorMap* m, const void* base, int E, int d, int f, int size, int kc) {
  const cuuint64_t row = static_cast<cuuint64_t>(f) * size;
  const cuuint64_t dim[3] = {row / 4, static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(E)};
  const cuuint64_t stride[2] = {row, row * d};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(kc * size / 4), 16, 1};
  return encode_words(m, base, 3, dim, stride, box);
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
  constexpr int kSize = kW8 ? 1 : 2;
  const Plan up = make_plan(p, kW8, false), down = make_plan(p, kW8, true);
  Maps m_up, m_down;
  if (!map_up(&m_up.routed, p.routed.gate_up, p.E, p.f, p.d, kSize, up.kc_d) ||
      !map_down(&m_down.routed, p.routed.down, p.E, p.d, p.f, kSize, down.kc_f))
    return false;
  if (p.fs && (!map_up(&m_up.shared, p.shared.gate_up, 1, p.fs, p.d, kSize, up.kc_d) ||
               !map_down(&m_down.shared, p.shared.down, 1, p.d, p.fs, kSize, down.kc_fs)))
    return false;
  // every CTA the same number of units, as far as the picked experts are known here: two CTAs an SM
  const int units = up.slots * (p.f / 8) + p.fs / 8, rounds = divide_up(units, 2 * sms);
  if (!launch(k_layer_up<kBf16, kW8, kNt>, divide_up(units, rounds), up, 1, s, m_up, p, up)) return false;
  const int blocks = p.d / 16, chunks = down.slots * divide_up(p.f, down.kc_f) + (p.fs ? divide_up(p.fs, down.kc_fs) : 0);
  int split = 1;
  while (split < 8 && 2 * split * blocks <= 2 * sms && 2 * split <= chunks) split *= 2;
  return launch(k_layer_down<kBf16, kW8, kNt>, blocks * split, down, split, s, m_down, p, down, split);
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
