// C entry points of the 16-bit operators: argument checks, then the launches
// (grouped_mm.cu, gated_lora.cu).  No context, no allocation, no state but the
// count of waits that ran out, which moe_grouped_sync reads.
#include "grouped.h"
#include "internal.h"
#include "op_checks.h"

namespace {

using namespace moe;

constexpr int kMaxRank = 128;
constexpr int kManyRows = 256;   // adapters: from here on their down half runs on tcgen05

bool side_ok(int v) { return v >= 8 && v <= kMaxSide && v % 8 == 0; }

bool groups_ok(int dtype, const int32_t* offsets, int n_experts, int m) {
  return (dtype == MOE_BF16 || dtype == MOE_F16) && offsets && aligned(offsets, 4) && n_experts >= 1 &&
         n_experts <= kMaxExperts && m >= 0 && m <= kMaxRows;
}

}  // namespace

extern "C" moe_status moe_grouped_mm(int dtype, int transpose, const void* x, int64_t ldx, int m, const int32_t* offsets,
                                     int n_experts, const void* w, int n, int k, void* y, int64_t ldy, int out_dtype,
                                     void* stream) {
  if (!groups_ok(dtype, offsets, n_experts, m) || !side_ok(n) || !side_ok(k)) return MOE_EINVAL;
  if (transpose != 0 && transpose != 1) return MOE_EINVAL;
  if (out_dtype != dtype && out_dtype != MOE_F32) return MOE_EINVAL;
  if (!w || !aligned(w, 16) || !rows_ok(x, m, ldx, transpose ? n : k) || !rows_ok(y, m, ldy, transpose ? k : n))
    return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  moe::GmOperands o;
  o.x = x, o.ldx = ldx, o.w = w, o.n = n, o.k = k;
  moe::GmParams p;
  p.offsets = offsets, p.E = n_experts, p.m = m;
  p.feat = transpose ? k : n, p.red = transpose ? n : k;
  p.y = y, p.ldy = ldy, p.out_f32 = out_dtype == MOE_F32, p.bf16 = dtype == MOE_BF16;
  return status(moe::launch_grouped(transpose ? moe::GM_DGRAD : moe::GM_FWD, moe::GM_PLAIN, o, p,
                                    static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_grouped_wgrad(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx, int m,
                                        const int32_t* offsets, int n_experts, int n, int k, void* dw, int out_dtype,
                                        void* stream) {
  if (!groups_ok(dtype, offsets, n_experts, m) || !side_ok(n) || !side_ok(k)) return MOE_EINVAL;
  if (out_dtype != dtype && out_dtype != MOE_F32) return MOE_EINVAL;
  if (!dw || !aligned(dw, 16) || !rows_ok(dy, m, lddy, n) || !rows_ok(x, m, ldx, k)) return MOE_EINVAL;
  if (m == 0) {
    const size_t bytes = static_cast<size_t>(n_experts) * n * k * (out_dtype == MOE_F32 ? 4 : 2);
    return status(cudaMemsetAsync(dw, 0, bytes, static_cast<cudaStream_t>(stream)) == cudaSuccess);
  }
  moe::GmOperands o;
  o.x = x, o.ldx = ldx, o.w = dy, o.ldw = lddy, o.n = n, o.k = k;
  moe::GmParams p;
  p.offsets = offsets, p.E = n_experts, p.m = m;
  p.feat = k, p.cols = n;
  p.y = dw, p.ldy = k, p.out_f32 = out_dtype == MOE_F32, p.bf16 = dtype == MOE_BF16;
  return status(moe::launch_grouped(moe::GM_WGRAD, moe::GM_PLAIN, o, p, static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_grouped_geglu(int dtype, int gelu_variant, const void* x, int64_t ldx, int m,
                                        const int32_t* offsets, int n_experts, const void* w, int f, int k, void* a,
                                        int64_t lda, void* h, int64_t ldh, void* stream) {
  if (!groups_ok(dtype, offsets, n_experts, m) || !gelu_ok(gelu_variant)) return MOE_EINVAL;
  if (f < 16 || f % 16 || f > kMaxSide / 2 || !side_ok(k)) return MOE_EINVAL;
  if (!w || !aligned(w, 16) || !rows_ok(x, m, ldx, k) || !rows_ok(a, m, lda, f)) return MOE_EINVAL;
  if (h && !rows_ok(h, m, ldh, 2 * static_cast<int64_t>(f))) return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  moe::GmOperands o;
  o.x = x, o.ldx = ldx, o.w = w, o.n = 2 * f, o.k = k;
  moe::GmParams p;
  p.offsets = offsets, p.E = n_experts, p.m = m;
  p.feat = f, p.red = k;
  p.y = a, p.ldy = lda, p.bf16 = dtype == MOE_BF16;
  p.h = h, p.ldh = ldh, p.gelu = gelu_variant;
  return status(moe::launch_grouped(moe::GM_FWD, moe::GM_GATED, o, p, static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_geglu_grad(int dtype, int gelu_variant, const void* h, int64_t ldh, const void* da,
                                     int64_t ldda, int m, int f, const int32_t* n_rows, void* dh, int64_t lddh,
                                     void* stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_F16) || !gelu_ok(gelu_variant)) return MOE_EINVAL;
  if (m < 0 || m > kMaxRows || f < 8 || f % 8 || f > kMaxSide / 2 || !aligned(n_rows, 4)) return MOE_EINVAL;
  if (!rows_ok(h, m, ldh, 2 * static_cast<int64_t>(f)) || !rows_ok(da, m, ldda, f) ||
      !rows_ok(dh, m, lddh, 2 * static_cast<int64_t>(f)))
    return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  return status(moe::launch_gated_grad(dtype == MOE_BF16, gelu_variant, h, ldh, da, ldda, dh, lddh, m, f, n_rows,
                                       static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_lora_mm(int dtype, const void* x, int64_t ldx, int t, const void* w, int n, int k,
                                  const int32_t* ids, const void* a, const void* b, const float* scale, int n_adapters,
                                  int rank, void* y, int64_t ldy, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
  if ((dtype != MOE_BF16 && dtype != MOE_F16) || t < 0 || t > kMaxRows || !side_ok(n) || !side_ok(k)) return MOE_EINVAL;
  if (n_adapters < 1 || rank < 8 || rank > kMaxRank || rank % 8) return MOE_EINVAL;
  if (!w || !a || !b || (!ids && t > 0) || !scale || !aligned(w, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(ids, 4) ||
      !aligned(scale, 4) || !rows_ok(x, t, ldx, k) || !rows_ok(y, t, ldy, n))
    return MOE_EINVAL;
  if ((!workspace && t > 0) || !aligned(workspace, 32) || workspace_bytes < static_cast<uint64_t>(t) * rank * 4) return MOE_EINVAL;
  if (t == 0) return MOE_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MOE_BF16;
  float* u = static_cast<float*>(workspace);
  moe::GmOperands o;
  o.x = x, o.ldx = ldx, o.w = a, o.n = n, o.k = k;
  moe::GmParams p;
  p.m = t, p.feat = n, p.red = k;
  p.y = y, p.ldy = ldy, p.bf16 = bf16;
  p.ids = ids, p.b = static_cast<const uint16_t*>(b), p.u = u, p.rank = rank, p.n_adapters = n_adapters;
  if (t >= kManyRows ? !moe::launch_adapter_down_many(o, p, scale, u, s)
                     : !moe::launch_adapter_down(bf16, x, ldx, t, a, scale, ids, n_adapters, rank, k, u, s))
    return MOE_ECUDA;
  o.w = w;
  return status(moe::launch_grouped(moe::GM_FWD, moe::GM_ADAPT, o, p, s));
}

extern "C" moe_status moe_grouped_sync(void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return MOE_ECUDA;
  if (capture != cudaStreamCaptureStatusNone) return MOE_EINVAL;
  bool news = false;
  if (!moe::grouped_gave_up(s, &news)) return MOE_ECUDA;
  return news ? MOE_ETIMEOUT : MOE_OK;
}
